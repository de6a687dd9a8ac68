"""The operators of a serving step over a paged cache: plan, rotary positions,
append and gather, and attention over the block-scaled 8-bit cache, each against
its plain 64-bit form; then a run of them together. The refusals at the end run
without a GPU."""
import ctypes
import math
import os
import subprocess
import sys
import tempfile

import pytest
import torch

from tests import paged_cache_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.finfo(torch.bfloat16).eps / 2
gpu = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32)


def _within(got, want, tol, what):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: pattern of finite values"
    f = torch.isfinite(want)
    over = ((got - want).abs() - tol)[f]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: {int((over > 0).sum())} over by up to {float(over.max()):.3g}"


# ---------------------------------------------------------------------------- plan


def _plan_case(batch, seed, most=40, context=100, idle=4):
    g = _gen(seed)
    seq = torch.randint(0, context + 1, (batch,), generator=g)
    new = torch.randint(0, most + 1, (batch,), generator=g) * (torch.randint(0, idle, (batch,), generator=g) > 0)
    width = (context + most + 15) // 16
    pages = torch.randperm(batch * (width + (most + 15) // 16 + 1) + 7, generator=g).to(torch.int32)
    table = pages[: batch * width].reshape(batch, width).clone()
    held = torch.arange(width)[None, :] < ((seq + 15) // 16)[:, None]
    table[~held] = -7
    return _i32(seq), _i32(new), table, pages[batch * width:].contiguous(), pages.numel()


@gpu
@pytest.mark.parametrize("batch,most,context", [(1, 1, 0), (1, 40, 15), (3, 1, 16), (64, 1, 500), (17, 40, 100),
                                                (300, 33, 64), (2500, 3, 40), (5, 3000, 31)])
def test_plan_matches_token_by_token(lib, batch, most, context):
    seq, new, table, free, blocks = _plan_case(batch, 3 + batch, most, context)
    total = int(new.sum()) + 5
    want = ref.plan_ref(seq, new, table, free, 2, total, None)
    d = [t.cuda() for t in (seq, new, table, free, _i32([2]))]
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = lib.plan_paged_step(*d, total, blocks, error_flags=flags)
    for name, a, b in zip(("lens", "cu", "positions", "slots", "used"), out, want):
        assert torch.equal(a.cpu(), b), name
    assert torch.equal(d[2].cpu(), want[5]) and int(flags.item()) == 0


@gpu
@pytest.mark.parametrize("batch,most,every", [(70, 25, 1), (2300, 1, 1), (2300, 1, 7), (2300, 2, 9), (512, 1, 1), (300, 40, 1),
                                              (2300, 5, 1)])
@pytest.mark.parametrize("in_place", [True, False])
def test_plan_advances_the_state(lib, batch, most, every, in_place):
    """Up to 512 rows, up to 2048 and above; more requests than one scan holds, most of them idle; over the old state."""
    seq, new, table, free, blocks = _plan_case(batch, 40 + batch, most, 33)
    new[torch.arange(batch) % every != 0] = 0
    total = int(new.sum()) + 2
    for clip in (0, 9):  # and with fewer rows than tokens
        fit = torch.minimum(new, (total - clip - (torch.cumsum(new, 0) - new)).clamp_min(0)).to(torch.int32)
        want = ref.plan_ref(seq, fit, table, free, 1, total - clip, None)
        d = [t.cuda() for t in (seq, new, table, free, _i32([1]))]
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        over = dict(seq_lens_out=d[0], num_used_out=d[4]) if in_place else {}
        out = lib.plan_paged_step(*d, total - clip, blocks, error_flags=flags, **over)
        for name, x, y in zip(("lens", "cu", "positions", "slots", "used"), out, want):
            assert torch.equal(x.cpu(), y), name
        assert torch.equal(d[2].cpu(), want[5]) and int(flags.item()) == (lib.ATTN_FAULT_BAD_LENGTH if clip else 0)


@gpu
def test_plan_advances_in_place_and_replays(lib):
    """Captured once and replayed, the state buffers carry over from step to step."""
    seq, new, table, free, blocks = _plan_case(9, 5, 20, 50)
    total = int(new.sum()) + 3
    d = [t.cuda() for t in (seq, new, torch.nn.functional.pad(table, (0, 4), value=-7), free, _i32([0]))]
    state = [d[0].clone(), d[2].clone(), d[4].clone()]
    pos, slots = torch.empty(total, dtype=torch.int32, device="cuda"), torch.empty(total, dtype=torch.int32, device="cuda")
    cu = torch.empty(10, dtype=torch.int32, device="cuda")

    def step():
        lib.plan_paged_step(d[0], d[1], d[2], d[3], d[4], total, blocks, seq_lens_out=d[0], cu_seqlens_q=cu,
                            positions=pos, slot_map=slots, num_used_out=d[4])
    step()
    torch.cuda.synchronize()
    for t, s in zip((d[0], d[2], d[4]), state):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    want = (seq, None, None, None, _i32([0]), torch.nn.functional.pad(table, (0, 4), value=-7))
    for _ in range(3):
        graph.replay()
        want = ref.plan_ref(want[0], new, want[5], free, int(want[4]), total, None)
        for a, b in ((d[0], want[0]), (cu, want[1]), (pos, want[2]), (slots, want[3]), (d[4], want[4]), (d[2], want[5])):
            assert torch.equal(a.cpu(), b)


@gpu
def test_plan_faults_are_flagged_and_bounded(lib):
    def run(seq, new, table, free, used, total, blocks):
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        table = table.cuda()
        out = lib.plan_paged_step(_i32(seq).cuda(), _i32(new).cuda(), table, _i32(free).cuda(), _i32([used]).cuda(), total,
                                  blocks, error_flags=flags)
        return int(flags.item()), [t.cpu().tolist() for t in out], table.cpu()
    empty = torch.full((2, 2), -1, dtype=torch.int32)
    # the free list runs out: the second sequence's token has no slot
    f, out, table = run([0, 0], [16, 1], empty, [4], 0, 17, 8)
    assert f == lib.ATTN_FAULT_NO_BLOCK and out[3] == list(range(64, 80)) + [-1] and out[4] == [1]
    assert table[1].tolist() == [-1, -1]
    # an id outside the pool
    f, out, _ = run([0, 0], [1, 0], empty, [9], 0, 1, 8)
    assert f == lib.ATTN_FAULT_BAD_BLOCK and out[3] == [-1]
    # past the table row: 32 tokens fit
    f, out, _ = run([30, -3], [5, 0], _i32([[1, 2], [3, 4]]), [5, 6], 0, 5, 8)
    assert f == lib.ATTN_FAULT_BAD_LENGTH and out[0] == [32, 0] and out[1] == [0, 2, 2] and out[3] == [46, 47, -1, -1, -1]
    # more new tokens than rows: what has no row takes no block and does not count
    f, out, _ = run([0, 0], [17, 17], empty, [5, 6, 7], 0, 20, 8)
    assert f == lib.ATTN_FAULT_BAD_LENGTH and out[0] == [17, 3] and out[1] == [0, 17, 20] and out[4] == [3]
    # nothing at all
    f, out, _ = run([0, 0], [0, 0], empty, [5], 0, 0, 8)
    assert f == 0 and out[1] == [0, 0, 0] and out[4] == [0]


# ---------------------------------------------------------------------------- rotary


@gpu
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(128, 128), (64, 64), (128, 32), (64, 48), (64, 16)])
@pytest.mark.parametrize("fin,fout", [("bfloat16", "bfloat16"), ("float32", "float32"), ("float32", "bfloat16"),
                                      ("bfloat16", "float32")])
def test_rotary_matches_definition(lib, packed, interleaved, D, R, fin, fout):
    g = _gen(D + R)
    B, S, Hq, Hk, mag = (1, 37, 6, 2, 1.25) if packed else (3, 13, 5, 5, 1.0)
    shape = (lambda h: (S, h, D)) if packed else (lambda h: (B, h, S, D))
    q, k = (torch.randn(shape(h), generator=g).to(getattr(torch, fin)) for h in (Hq, Hk))
    pos = torch.randint(0, 1000000, (S,) if packed else (B, S), generator=g).to(torch.int32)
    pos.view(-1)[3] = 0
    freq = ref.frequencies(R)
    for inverse in (False, True):
        out = lib.rotary(q.cuda(), k.cuda(), freq.cuda(), pos.cuda(), interleaved=interleaved, inverse=inverse,
                         magnitude=mag, out_dtype=getattr(torch, fout))
        for x, y in zip((q, k), out):
            p = pos[:, None] if packed else pos[:, None, :]
            want, size = ref.rotate_ref(x.double(), p, freq, mag, interleaved, inverse)
            rounding = torch.finfo(getattr(torch, fout)).eps / 2
            _within(y, want, size * ref.TURN_REL + want.abs() * rounding * 1.001, "turned")


@gpu
def test_rotary_defaults_strides_in_place_and_skipped_rows(lib):
    g = _gen(1)
    B, S, H, D = 2, 70, 3, 64
    freq = ref.frequencies(D)
    base = torch.randn(B, S, 2 * H + 1, D, generator=g).to(torch.bfloat16).cuda()  # rows of a projection
    q = base.transpose(1, 2)[:, :H]
    want, size = ref.rotate_ref(q.double().cpu(), torch.arange(S)[None, None, :], freq)
    out, none = lib.rotary(q, None, freq.cuda())
    assert none is None
    _within(out, want, size * ref.TURN_REL + want.abs() * BF16 * 1.001, "default positions")
    pos = torch.arange(S, dtype=torch.int32).repeat(B, 1)
    pos[1, 50:] = -1
    kept = base.clone()
    lib.rotary(q, None, freq.cuda(), pos.cuda(), q_out=q)  # in place
    torch.cuda.synchronize()
    assert torch.equal(q[0], out[0]) and torch.equal(q[1, :, :50], out[1, :, :50])
    assert torch.equal(base[1, 50:], kept[1, 50:]) and torch.equal(base[:, :, H:], kept[:, :, H:])


@gpu
def test_rotary_gradient_against_differences(lib):
    """The map is linear: <turn(x + d) - turn(x), w> = <d, inverse turn(w)> up to fp32 rounding."""
    g = _gen(2)
    S, H, D, mag = 33, 2, 128, 0.75
    freq = ref.frequencies(64).cuda()
    x, d, w = (torch.randn(S, H, D, generator=g).cuda() for _ in range(3))
    pos = torch.randint(0, 5000, (S,), generator=g).to(torch.int32).cuda()
    f = lambda t, inv=False: lib.rotary(t, None, freq, pos, magnitude=mag, inverse=inv)[0].double()  # noqa: E731
    diff = ((f(x + d) - f(x)) * w.double()).sum()
    grad = (d.double() * f(w, True)).sum()
    # every product's terms are off by at most 2^-20 of their sizes: x + d and three turns
    size = ((x.abs() + d.abs()).double().amax() * 4 * w.double().abs()).sum()
    assert abs(float(diff - grad)) <= 2.0 ** -20 * float(size)


@gpu
def test_rotary_far_positions(lib):
    """Close to 2^31 the angle keeps its remainder: p * f / pi is off by 2.5 * 2^-53 of 2^29.4 half turns, 2^-20.6 rad,
    and the 64-bit form by 2^-22 rad."""
    pos = torch.tensor([2 ** 31 - 1, 2 ** 31 - 1000, 2 ** 30 + 1], dtype=torch.int32)
    freq = ref.frequencies(64)
    x = torch.randn(3, 2, 64, generator=_gen(3))
    y, _ = lib.rotary(x.cuda(), None, freq.cuda(), pos.cuda())
    want, size = ref.rotate_ref(x.double(), pos[:, None], freq)
    _within(y, want, size * (ref.TURN_REL + 2.0 ** -20), "far")


# ---------------------------------------------------------------------------- append and gather


def _append_case(old, new, Hq, Hk, D, fp8, seed):
    g = _gen(seed)
    old, new = torch.tensor(old), torch.tensor(new)
    lens = old + new
    table, nb = ref.tables(g, lens, int((lens.max() + 15) // 16) + 1)
    if fp8:
        kc, ks = ref.random_cache(g, nb, Hk, D, table, old)
        vc, vs = ref.random_cache(g, nb, Hk, D, table, old)
    else:
        kc, vc = (torch.randn(nb, Hk, 16, D, generator=g).to(torch.bfloat16) for _ in range(2))
        ks = vs = None
    seq = torch.repeat_interleave(torch.arange(len(old)), new)
    first = torch.cumsum(new, 0) - new
    pos = old[seq] + torch.arange(seq.numel()) - first[seq]
    slots = table[seq, pos // 16] * 16 + (pos % 16).to(torch.int32)
    rows = torch.randn(seq.numel(), Hq + 2 * Hk, D, generator=g).to(torch.bfloat16)
    return dict(old=old, new=new, lens=lens, table=table, nb=nb, kc=kc, vc=vc, ks=ks, vs=vs, pos=pos.to(torch.int32),
                slots=slots.to(torch.int32), q=rows[:, :Hq], k=rows[:, Hq:Hq + Hk], v=rows[:, Hq + Hk:])


def _run_append(lib, c, freq, mag, interleaved, with_q=True):
    dev = {n: (None if t is None else t.cuda()) for n, t in c.items() if isinstance(t, torch.Tensor) or t is None}
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = lib.append_paged(dev["k"], dev["v"], dev["slots"], dev["kc"], dev["vc"], dev["ks"], dev["vs"],
                         q=dev["q"] if with_q else None, inv_freq=None if freq is None else freq.cuda(),
                         positions=None if freq is None else dev["pos"], interleaved=interleaved, magnitude=mag,
                         error_flags=flags)
    torch.cuda.synchronize()
    return q, dev, int(flags.item())


def _check_pages(c, dev, name, want, size):
    """Pages after an append of FP8 rows `want` [T, H, D] (64 bits, each off by `size`) against the definition."""
    codes0, scales0 = c[name + "c"], c[name + "s"]
    codes, scales = dev[name + "c"].cpu(), dev[name + "s"].cpu()
    before, after = ref.values(codes0, scales0), ref.values(codes, scales)
    touched = {}
    for t, slot in enumerate(c["slots"].tolist()):
        if slot >= 0:
            touched.setdefault(slot // 16, []).append((slot % 16, t))
    for blk in range(c["nb"]):
        if blk not in touched:
            assert torch.equal(codes[blk], codes0[blk]) and torch.equal(scales[blk], scales0[blk])
            continue
        off0, end = touched[blk][0][0], touched[blk][-1][0] + 1
        rows = [t for _, t in touched[blk]]
        assert torch.equal(codes[blk, :, end:], codes0[blk, :, end:])
        kept = before[blk, :, :off0]
        new = want[rows].transpose(0, 1)
        off = size[rows].transpose(0, 1)
        for h in range(codes.shape[1]):
            full = torch.cat((kept[h], new[h]))
            e = int(scales[blk, h]) - 127
            finite = full[torch.isfinite(full)]
            top, slack = float(finite.abs().max()) if finite.numel() else 0.0, float(off[h].nan_to_num(0).max())
            assert ref.exponent(max(0.0, top - slack)) <= e <= ref.exponent(top + slack), (blk, h, e, top)
            # half a step of E4M3: 2^-4 of the value, 2^-10 of the scale where codes are subnormal
            half = torch.maximum(full.abs() * 2.0 ** -4, torch.full_like(full, 2.0 ** (e - 10)))
            half[:off0] = torch.where(full[:off0].abs() >= 2.0 ** (e - 6), 0.0, 2.0 ** (e - 10))  # kept: exact while normal
            half[off0:] += off[h] * 2
            _within(after[blk, h, :end], torch.where(torch.isfinite(full), full, math.nan), half, f"{name} block {blk}")


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("old,new", [([0], [1]), ([15, 16, 17, 3], [1, 1, 1, 1]), ([5, 0, 31, 700], [40, 16, 1, 200]),
                                     ([0, 1, 2, 3, 15], [0, 31, 30, 13, 17]), ([7] * 90, [1] * 90)])
def test_append_fp8_matches_definition(lib, D, interleaved, old, new):
    c = _append_case(old, new, 6, 3, D, True, 11)
    freq, mag = ref.frequencies(D // 2), 1.5
    q, dev, flags = _run_append(lib, c, freq, mag, interleaved)
    assert flags == 0
    turn = lambda x: ref.rotate_ref(x.double(), c["pos"][:, None], freq, mag, interleaved)  # noqa: E731
    want, size = turn(c["q"])
    _within(q, want, size * ref.TURN_REL + want.abs() * BF16 * 1.001, "q")
    want, size = turn(c["k"])
    _check_pages(c, dev, "k", want, size * ref.TURN_REL)
    _check_pages(c, dev, "v", c["v"].double(), torch.zeros_like(c["v"], dtype=torch.float64))
    width = int(c["lens"].max()) + 3
    dk, dv = lib.gather_paged(dev["kc"], dev["vc"], dev["table"], _i32(c["lens"]).cuda(), width, dev["ks"], dev["vs"])
    for got, name in ((dk, "k"), (dv, "v")):
        vals = ref.values(dev[name + "c"].cpu(), dev[name + "s"].cpu())
        assert torch.equal(got.double().cpu(), ref.dense(vals, c["table"], c["lens"], width))


@gpu
@pytest.mark.parametrize("new,Hk", [([1, 40, 16], 1), ([300, 33, 700], 5), ([2000, 1200, 1600], 20)])
def test_append_shares_heads_out(lib, new, Hk):
    """One CTA for all heads of K and V, CTAs of either, and CTAs that hold the last heads of K and the first of V."""
    c = _append_case([5, 0, 31], new, Hk, Hk, 64, True, 16)
    freq = ref.frequencies(64)
    q, dev, flags = _run_append(lib, c, freq, 1.0, False)
    assert flags == 0
    turn = lambda x: ref.rotate_ref(x.double(), c["pos"][:, None], freq)  # noqa: E731
    want, size = turn(c["q"])
    _within(q, want, size * ref.TURN_REL + want.abs() * BF16 * 1.001, "q")
    want, size = turn(c["k"])
    _check_pages(c, dev, "k", want, size * ref.TURN_REL)
    _check_pages(c, dev, "v", c["v"].double(), torch.zeros_like(c["v"], dtype=torch.float64))


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_append_bf16_any_order(lib, D):
    c = _append_case([5, 0, 31], [40, 16, 1], 4, 2, D, False, 12)
    order = torch.randperm(c["slots"].numel(), generator=_gen(13))
    for n in ("q", "k", "v", "pos", "slots"):
        c[n] = c[n][order]
    freq = ref.frequencies(D)
    q, dev, flags = _run_append(lib, c, freq, 1.0, False)
    assert flags == 0
    want, size = ref.rotate_ref(c["k"].double(), c["pos"][:, None], freq)
    blk, off = (c["slots"] // 16).long(), (c["slots"] % 16).long()
    _within(dev["kc"].cpu()[blk, :, off], want, size * ref.TURN_REL + want.abs() * BF16 * 1.001, "k")
    expect = c["vc"].clone()
    expect[blk, :, off] = c["v"]
    assert torch.equal(dev["vc"].cpu(), expect)
    width = 60
    dk, dv = lib.gather_paged(dev["kc"], dev["vc"], dev["table"], _i32(c["lens"]).cuda(), width)
    assert torch.equal(dv.double().cpu(), ref.dense(expect.double(), c["table"], c["lens"], width))
    assert torch.equal(dk.double().cpu(), ref.dense(dev["kc"].cpu().double(), c["table"], c["lens"], width))


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_append_skips_padding_and_flags_bad_slots(lib, fp8):
    c = _append_case([3, 20], [6, 4], 4, 2, 64, fp8, 14)
    whole = _run_append(lib, dict(c), None, 1.0, False)[1]
    c["slots"] = torch.cat((c["slots"], _i32([-1, c["nb"] * 16, 2 ** 31 - 1, -2 ** 31])))
    for n in ("q", "k", "v"):
        c[n] = torch.cat((c[n], torch.full_like(c[n][:4], math.nan)))
    c["pos"] = torch.cat((c["pos"], _i32([-1, -1, -1, -1])))
    q, dev, flags = _run_append(lib, c, None, 1.0, False)
    assert flags == lib.ATTN_FAULT_BAD_BLOCK
    for n in ("kc", "vc", "ks", "vs"):
        assert (dev[n] is None and whole[n] is None) or torch.equal(dev[n], whole[n])
    assert torch.equal(q[:10].cpu(), c["q"][:10])


@gpu
def test_append_fp8_special_values(lib):
    """NaN and infinities are stored as NaN and leave the scale alone; zeros; the largest and smallest magnitudes."""
    c = _append_case([0, 0, 0, 0], [16, 3, 16, 2], 2, 1, 64, True, 15)
    v, k = c["v"].clone(), c["k"].clone()
    v[2, 0, 5], v[3, 0, 6], v[4, 0, 7] = math.inf, -math.inf, math.nan
    v[16:19] = 0.0
    v[19:35] *= 2.0 ** 100
    v[35:37] *= 2.0 ** -120
    k[0] = math.nan
    c["v"], c["k"] = v, k
    _, dev, flags = _run_append(lib, c, None, 1.0, False, with_q=False)
    assert flags == 0
    zero = torch.zeros_like(v, dtype=torch.float64)
    _check_pages(c, dev, "v", torch.where(torch.isfinite(v), v, math.nan).double(), zero)
    _check_pages(c, dev, "k", k.double(), zero)


# ---------------------------------------------------------------------------- attention over the block-scaled cache


def _attention_tol(q, k, scales_of_v, v, scale, limit, weight_step, tiny_step):
    """Reference and tolerances of one kv head's rows.

    Scores: a dot product of D terms in fp32 is off by at most D 2^-24 of the sum
    of its terms' sizes, and scaling and exponential add less than 2^-20; a score
    off by d changes a weight and the row's sum by a factor of at most e^d each.
    Weights are rounded by weight_step, relative, before the product with V; in
    fp16 (tiny_step) a weight below 2^-14 of the largest is off by 2^-25 of it.
    """
    o, lse, pv, size, p = ref.attend_ref(q, k, v, scale, limit)
    d = size * (q.shape[-1] * 2.0 ** -24) + 2.0 ** -20 * (1 + size)
    tol = (torch.expm1(2 * d) + weight_step)[..., None] * pv
    if tiny_step:
        w = p * torch.exp2(scales_of_v)[:, None, :]
        tol = tol + tiny_step * w.amax(-1, keepdim=True) * (v.abs() / torch.exp2(scales_of_v)[..., None]).sum(1)[:, None]
    return o, lse, tol, d + 2.0 ** -20 * (1 + torch.where(torch.isinf(lse), 0.0, lse).abs())


def _decode_case(lens, Hq, Hk, D, seed, spread=3.0):
    g = _gen(seed)
    table, nb = ref.tables(g, lens, (max(lens) + 15) // 16 + 1)
    kc, ks = ref.random_cache(g, nb, Hk, D, table, lens, spread)
    vc, vs = ref.random_cache(g, nb, Hk, D, table, lens, spread)
    q = torch.randn(len(lens), Hq, D, generator=g).to(torch.bfloat16)
    return dict(lens=list(lens), table=table, kc=kc, ks=ks, vc=vc, vs=vs, q=q, Hq=Hq, Hk=Hk, D=D, scale=D ** -0.5)


def _decode_want(c):
    B, G = len(c["lens"]), c["Hq"] // c["Hk"]
    kv, vv = ref.values(c["kc"], c["ks"]), ref.values(c["vc"], c["vs"])
    outs = []
    for b, n in enumerate(c["lens"]):
        ids = c["table"][b, : (n + 15) // 16].long()
        k, v = (x[ids].transpose(0, 1).reshape(c["Hk"], -1, c["D"])[:, :n] for x in (kv, vv))
        ev = (c["vs"][ids].double() - 127).T.repeat_interleave(16, 1)[:, :n]
        q = c["q"][b].double().reshape(c["Hk"], G, c["D"])
        outs.append(_attention_tol(q, k, ev, v, c["scale"], torch.full((G,), n), 2.0 ** -11, 2.0 ** -25 if n else 0))
    cat = lambda i, shape: torch.stack([o[i].reshape(shape) for o in outs])  # noqa: E731
    o, tol = cat(0, (c["Hq"], c["D"])), cat(2, (c["Hq"], c["D"]))
    return o, cat(1, (c["Hq"],)), tol, cat(3, (c["Hq"],))


def _decode_run(lib, c, **kw):
    dev = {n: c[n].cuda() for n in ("q", "kc", "vc", "ks", "vs", "table")}
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = lib.decode_paged_block_scaled(dev["q"], dev["kc"], dev["vc"], dev["ks"], dev["vs"], dev["table"],
                                           _i32(c["lens"]).cuda(), c["scale"], error_flags=flags, **kw)
    torch.cuda.synchronize()
    return o, lse, int(flags.item())


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 4, 8, 9, 16])
@pytest.mark.parametrize("num_splits", [0, 1, 5, 16])
def test_decode_block_scaled_matches_definition(lib, D, G, num_splits):
    c = _decode_case([1, 0, 15, 16, 17, 100, 643, 2500], 2 * G, 2, D, 100 + G)
    o, lse, tol, ltol = _decode_want(c)
    for dtype in (torch.float32, torch.bfloat16):
        go, gl, flags = _decode_run(lib, c, num_splits=num_splits, out_dtype=dtype, max_seq_len=max(c["lens"]))
        assert flags == 0
        _within(go, o, tol + 2.0 ** -21 * o.abs() + (o.abs() * BF16 * 1.01 if dtype == torch.bfloat16 else 0), "O")
        _within(gl, lse, ltol, "LSE")
    assert (go[1] == 0).all() and torch.isneginf(gl[1]).all()


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [4, 12])
@pytest.mark.parametrize("batch,num_splits", [(2, 4), (2, 16), (40, 2), (40, 8), (6, 32)])
def test_decode_block_scaled_small_and_large_grids(lib, D, G, batch, num_splits):
    """Grids below one CTA per SM and above it, as one cluster and as several, with and without keys for every CTA."""
    c = _decode_case(([4200, 130, 700, 1, 0, 257] + [40 + 31 * i for i in range(34)])[:batch], 2 * G, 2, D, 300 + G)
    o, lse, tol, ltol = _decode_want(c)
    go, gl, flags = _decode_run(lib, c, num_splits=num_splits, out_dtype=torch.float32, max_seq_len=max(c["lens"]))
    assert flags == 0
    _within(go, o, tol + 2.0 ** -21 * o.abs(), "O")
    _within(gl, lse, ltol, "LSE")


@gpu
@pytest.mark.parametrize("spread", [0.0, 30.0])
def test_decode_block_scaled_far_scales(lib, spread):
    """Blocks whose value scales lie up to 2^60 apart, keys near one scale; and a long sequence (many batches of blocks)."""
    c = _decode_case([3000, 40], 8, 2, 128, 5, 0.0)
    g = _gen(6)
    live = c["vs"] != 255
    shift = ((torch.rand(c["vs"].shape, generator=g) * 2 - 1) * spread).round().to(torch.int32)
    c["vs"] = torch.where(live, c["vs"].int() + shift, 255).to(torch.uint8)
    o, lse, tol, ltol = _decode_want(c)
    for n in (1, 0, 7, 16):
        go, gl, flags = _decode_run(lib, c, num_splits=n, out_dtype=torch.float32)
        assert flags == 0
        _within(go, o, tol + 2.0 ** -21 * o.abs(), f"O splits {n}")
        _within(gl, lse, ltol, "LSE")


@gpu
def test_decode_block_scaled_queries_of_any_size(lib):
    """Queries beyond fp16's range and far below it, and a zero query."""
    c = _decode_case([200, 33, 5], 4, 1, 128, 7, 0.0)
    c["q"][0] *= 2.0 ** 40
    c["q"][1] *= 2.0 ** -60
    c["q"][2, 0] = 0.0
    c["ks"] = torch.where(c["ks"] == 255, 255, c["ks"].int() - 44).to(torch.uint8)
    o, lse, tol, ltol = _decode_want(c)
    go, gl, _ = _decode_run(lib, c, out_dtype=torch.float32)
    _within(go, o, tol + 2.0 ** -21 * o.abs(), "O")
    _within(gl, lse, ltol, "LSE")


@gpu
def test_decode_block_scaled_nan_in_live_tokens(lib):
    c = _decode_case([40, 40, 40, 700], 4, 2, 64, 8)
    c["kc"][int(c["table"][0, 1]), 0, 3, 5] = 0x7F
    c["vs"][int(c["table"][1, 0]), 1] = 255
    c["vc"][int(c["table"][3, 30]), 1, 3, 9] = 0xFF
    for splits in (1, 3, 0):
        o, lse, _ = _decode_run(lib, c, num_splits=splits)
        o, lse = o.cpu(), lse.cpu()
        assert torch.isnan(o[0, :2]).all() and torch.isnan(lse[0, :2]).all() and torch.isfinite(o[0, 2:]).all()
        assert torch.isnan(o[1, 2:]).all() and torch.isfinite(o[1, :2]).all() and torch.isfinite(lse[1]).all()
        assert torch.isfinite(o[2]).all()
        nan = torch.zeros(4, 64, dtype=torch.bool)
        nan[2:, 9] = True
        assert torch.equal(torch.isnan(o[3]), nan)


@gpu
def test_decode_block_scaled_bad_tables_and_lengths(lib):
    c = _decode_case([64, 64, 64], 4, 1, 64, 9)
    c["table"][1, 2] = 10 ** 6
    o, _, flags = _decode_run(lib, c)
    assert flags == lib.ATTN_FAULT_BAD_BLOCK and torch.isfinite(o).all()
    c["table"][1, 2] = c["table"][1, 1]
    want, _, tol, _ = _decode_want(c)
    c["lens"] = [64, 64, -5]
    o, lse, flags = _decode_run(lib, c, out_dtype=torch.float32)
    assert flags == lib.ATTN_FAULT_BAD_LENGTH and (o[2] == 0).all() and torch.isneginf(lse[2]).all()
    _within(o[:2], want[:2], tol[:2] + 2.0 ** -21 * want[:2].abs(), "others")
    c["lens"] = [64, 64, 64]
    o, lse, flags = _decode_run(lib, c, max_seq_len=30, num_splits=1)  # cut at the plan's bound, flagged, no write outside
    assert torch.isfinite(o).all()


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(4, 2), (3, 1), (5, 5), (16, 2)])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("chunks,contexts", [([1, 1, 1], [0, 16, 700]), ([5, 0, 3, 16], [30, 5, 0, 129]),
                                             ([130, 7, 300], [0, 1000, 41])])
def test_prefill_block_scaled_matches_definition(lib, D, Hq, Hk, packed, chunks, contexts):
    g = _gen(sum(chunks) + D)
    B, G, most = len(chunks), Hq // Hk, max(chunks)
    lens = [a + b for a, b in zip(chunks, contexts)]
    c = _decode_case(lens, Hq, Hk, D, 17)
    dev = {n: c[n].cuda() for n in ("kc", "vc", "ks", "vs", "table")}
    q = torch.randn(sum(chunks), Hq, D, generator=g).to(torch.bfloat16)
    cu = _i32([0] + torch.cumsum(torch.tensor(chunks), 0).tolist())
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    for causal in (True, False):
        for dtype in (torch.float32, torch.bfloat16):
            kw = dict(scale=c["scale"], causal=causal, out_dtype=dtype, max_seqlen_k=max(lens), error_flags=flags)
            args = [dev[n] for n in ("kc", "vc", "ks", "vs", "table")] + [_i32(lens).cuda()]
            if packed:
                o, lse = lib.prefill_paged_block_scaled(q.cuda(), *args, cu_seqlens_q=cu.cuda(), max_seqlen_q=most, **kw)
            else:
                pad = torch.zeros(B, Hq, most, D, dtype=torch.bfloat16)
                for b in range(B):
                    pad[b, :, :chunks[b]] = q[cu[b]:cu[b + 1]].transpose(0, 1)
                out = torch.full(pad.shape, 7.0, dtype=dtype, device="cuda")
                o, lse = lib.prefill_paged_block_scaled(pad.cuda(), *args, seqlens_q=_i32(chunks).cuda(), out=out, **kw)
            torch.cuda.synchronize()
            kv, vv = ref.values(c["kc"], c["ks"]), ref.values(c["vc"], c["vs"])
            for b, n in enumerate(lens):
                ids = c["table"][b, : (n + 15) // 16].long()
                k, v = (x[ids].transpose(0, 1).reshape(Hk, -1, D)[:, :n] for x in (kv, vv))
                ev = (c["vs"][ids].double() - 127).T.repeat_interleave(16, 1)[:, :n]
                rows = chunks[b]
                if packed:
                    got, gl = o[cu[b]:cu[b + 1]].transpose(0, 1), lse[:, cu[b]:cu[b + 1]]
                else:
                    got, gl = o[b, :, :rows], lse[b, :, :rows]
                    assert (o[b, :, rows:] == 7.0).all()
                limit = torch.arange(n - rows + 1, n + 1) if causal else torch.full((rows,), n)
                qs = q[cu[b]:cu[b + 1]].double().permute(1, 0, 2).reshape(Hk, G * rows, D)
                want, wl, tol, ltol = _attention_tol(qs, k, ev, v, c["scale"], limit.repeat(G), 2.0 ** -8 + 2.0 ** -11, 0)
                want, tol = want.reshape(Hq, rows, D), tol.reshape(Hq, rows, D)
                rounding = want.abs() * BF16 * 1.01 if dtype == torch.bfloat16 else 0
                _within(got, want, tol + 2.0 ** -20 * want.abs() + rounding, f"O {b}")
                # the running sum is made of exponentials within 2^-12 of the exact ones
                _within(gl, wl.reshape(Hq, rows), ltol.reshape(Hq, rows) + 2.0 ** -12, f"LSE {b}")
    assert int(flags.item()) == 0


@gpu
def test_prefill_block_scaled_bounds_and_empty_rows(lib):
    c = _decode_case([40, 20], 4, 2, 64, 21)
    dev = [c[n].cuda() for n in ("kc", "vc", "ks", "vs", "table")]
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.randn(2, 4, 24, 64, generator=_gen(4)).to(torch.bfloat16).cuda()
    # 24 rows over 20 keys: the first 4 see nothing
    o, lse = lib.prefill_paged_block_scaled(q, *dev, _i32([40, 20]).cuda(), max_seqlen_k=40, error_flags=flags)
    assert (o[1, :, :4] == 0).all() and torch.isneginf(lse[1, :, :4]).all() and torch.isfinite(lse[1, :, 4:]).all()
    assert torch.isfinite(o).all() and int(flags.item()) == 0
    # a length over the caller's bound is cut and flagged
    o2, _ = lib.prefill_paged_block_scaled(q, *dev, _i32([40, 20]).cuda(), max_seqlen_k=33, causal=False, error_flags=flags)
    o3, _ = lib.prefill_paged_block_scaled(q, *dev, _i32([33, 20]).cuda(), max_seqlen_k=33, causal=False)
    assert int(flags.item()) == lib.ATTN_FAULT_BAD_LENGTH and torch.equal(o2, o3)
    # no keys at all
    o, lse = lib.prefill_paged_block_scaled(q, *dev, _i32([0, 0]).cuda(), max_seqlen_k=0)
    assert (o == 0).all() and torch.isneginf(lse).all()
    # the same for as many rows and keys as the tensor-core tiles are taken for
    c = _decode_case([900, 500], 16, 2, 128, 25)
    dev = [c[n].cuda() for n in ("kc", "vc", "ks", "vs", "table")]
    q = torch.randn(2, 16, 600, 128, generator=_gen(26)).to(torch.bfloat16).cuda()
    flags.zero_()
    o, lse = lib.prefill_paged_block_scaled(q, *dev, _i32([900, 500]).cuda(), max_seqlen_k=900, error_flags=flags)
    assert (o[1, :, :100] == 0).all() and torch.isneginf(lse[1, :, :100]).all() and torch.isfinite(lse[1, :, 100:]).all()
    assert torch.isfinite(o).all() and int(flags.item()) == 0
    o2, _ = lib.prefill_paged_block_scaled(q, *dev, _i32([900, -4]).cuda(), max_seqlen_k=833, causal=False, error_flags=flags)
    o3, _ = lib.prefill_paged_block_scaled(q, *dev, _i32([833, 0]).cuda(), max_seqlen_k=833, causal=False)
    assert int(flags.item()) == lib.ATTN_FAULT_BAD_LENGTH and torch.equal(o2, o3) and (o2[1] == 0).all()
    dev[4][0, 3] = 10 ** 6  # a page outside the pool: flagged, read as zeros
    o, _ = lib.prefill_paged_block_scaled(q, *dev, _i32([900, 500]).cuda(), max_seqlen_k=900, error_flags=flags)
    assert int(flags.item()) & lib.ATTN_FAULT_BAD_BLOCK and torch.isfinite(o).all()


@gpu
@pytest.mark.parametrize("rows,context,D,Hq", [(9, 20, 64, 4), (9, 1500, 64, 4), (512, 2000, 128, 8)])
def test_prefill_block_scaled_nan_in_a_visible_key(lib, rows, context, D, Hq):
    """Rows that see a NaN key give NaN (O and LSE), the rows before it and the other head do not.

    The last case has the rows and keys for which the tensor-core tiles are taken."""
    n, G = context + rows, Hq // 2
    for col in range(8):  # every place in a run of columns
        c = _decode_case([n], Hq, 2, D, 22)
        at = context + 1 + col % 8
        c["kc"][int(c["table"][0, at // 16]), 1, at % 16, 3] = 0x7F
        dev = [c[k].cuda() for k in ("kc", "vc", "ks", "vs", "table")]
        q = torch.randn(1, Hq, rows, D, generator=_gen(col)).to(torch.bfloat16).cuda()
        o, lse = lib.prefill_paged_block_scaled(q, *dev, _i32([n]).cuda(), max_seqlen_k=n)
        sees = torch.arange(context, n) >= at
        assert torch.isfinite(o[:, :G]).all() and torch.isfinite(lse[:, :G]).all()
        for h in range(G, Hq):
            assert torch.equal(torch.isnan(o[0, h]).all(-1).cpu(), sees) and torch.equal(torch.isnan(lse[0, h]).cpu(), sees)
            assert torch.isfinite(o[0, h][~sees]).all()


@gpu
@pytest.mark.parametrize("D,Hq,Hk,chunks", [(64, 4, 2, [1, 130, 3, 0]), (128, 8, 2, [300, 1, 77, 0]),
                                            (128, 3, 1, [300, 1, 77, 0]), (128, 16, 2, [40, 300, 3, 0]),
                                            (64, 24, 2, [300, 1, 3, 200])])
def test_prefill_block_scaled_shared_items(lib, D, Hq, Hk, chunks):
    """Chunks over long keys (all but the first for the tensor-core tiles, with 4, 1, 8 and 4 heads per tile): every
    item's keys are shared by many CTAs, and ragged lengths end inside shares."""
    lens = [6000, 4100, max(3, chunks[2]), 900]
    c = _decode_case(lens, Hq, Hk, D, 23)
    q = torch.randn(sum(chunks), Hq, D, generator=_gen(24)).to(torch.bfloat16)
    cu = [0] + torch.cumsum(torch.tensor(chunks), 0).tolist()
    dev = [c[k].cuda() for k in ("kc", "vc", "ks", "vs", "table")]
    runs = [lib.prefill_paged_block_scaled(q.cuda(), *dev, _i32(lens).cuda(), cu_seqlens_q=_i32(cu).cuda(), max_seqlen_q=max(chunks),
                                           out_dtype=torch.float32) for _ in range(2)]
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])  # no order of arrival in it
    kv, vv = ref.values(c["kc"], c["ks"]), ref.values(c["vc"], c["vs"])
    for b, n in enumerate(lens):
        rows = chunks[b]
        ids = c["table"][b, : (n + 15) // 16].long()
        k, v = (x[ids].transpose(0, 1).reshape(Hk, -1, D)[:, :n] for x in (kv, vv))
        ev = (c["vs"][ids].double() - 127).T.repeat_interleave(16, 1)[:, :n]
        qs = q[cu[b]:cu[b + 1]].double().permute(1, 0, 2).reshape(Hk, Hq // Hk * rows, D)
        limit = torch.arange(n - rows + 1, n + 1).repeat(Hq // Hk)
        want, wl, tol, ltol = _attention_tol(qs, k, ev, v, c["scale"], limit, 2.0 ** -8 + 2.0 ** -11, 0)
        got, gl = runs[0][0][cu[b]:cu[b + 1]].transpose(0, 1), runs[0][1][:, cu[b]:cu[b + 1]]
        _within(got, want.reshape(Hq, rows, D), tol.reshape(Hq, rows, D) + 2.0 ** -20 * want.reshape(Hq, rows, D).abs(), f"O {b}")
        _within(gl, wl.reshape(Hq, rows), ltol.reshape(Hq, rows) + 2.0 ** -12, f"LSE {b}")


# ---------------------------------------------------------------------------- what no case above does


@gpu
def test_offsets_past_32_bits(lib):
    """Pages in the last blocks of pools of more than 4 GiB (and scales, slots to match) give the same bits as near ones."""
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("needs 14 GiB of free device memory")
    Hk, Hq, D, nb = 8, 16, 128, (1 << 32) // (8 * 16 * 128) + 40
    g, new = _gen(41), 40
    qkv = torch.randn(new, Hq + 2 * Hk, D, generator=g).to(torch.bfloat16).cuda()
    freq, pos = ref.frequencies(64).cuda(), torch.arange(new, dtype=torch.int32, device="cuda")
    outs = []
    pools = [torch.empty(nb, Hk, 16, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((nb, Hk), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for ids in ([2, 0, 1], [nb - 1, nb - 7, nb - 3]):
        table = torch.tensor([ids], dtype=torch.int32, device="cuda")
        slots = table[0, (pos // 16).long()] * 16 + pos % 16
        args = (pools[0], pools[1], scales[0], scales[1])
        q = lib.append_paged(qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], slots, *args, q=qkv[:, :Hq], inv_freq=freq, positions=pos)
        lens = _i32([new]).cuda()
        k, v = lib.gather_paged(pools[0], pools[1], table, lens, new, *scales)
        o, lse = lib.decode_paged_block_scaled(q[-1:].contiguous(), *args, table, lens)
        p, _ = lib.prefill_paged_block_scaled(q, *args, table, lens, cu_seqlens_q=_i32([0, new]).cuda(), max_seqlen_q=new)
        big = qkv.new_zeros(1, 4 * Hq, 1024, D)  # many rows: the tensor-core path
        t, _ = lib.prefill_paged_block_scaled(big, *args, table, lens, causal=False)
        outs.append((q, k, v, o, lse, p, t))
    for a, b in zip(*outs):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@gpu
def test_empty_calls(lib):
    e = lambda *s, dtype=torch.int32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    out = lib.plan_paged_step(e(0), e(0), e(0, 4), e(0), _i32([0]).cuda(), 0, 9)
    assert out[1].tolist() == [0] and out[4].tolist() == [0]
    out = lib.plan_paged_step(e(0), e(0), e(0, 4), e(0), _i32([0]).cuda(), 3, 9)
    assert out[2].tolist() == [-1, -1, -1] and out[3].tolist() == [-1, -1, -1]
    bf = lambda *s: e(*s, dtype=torch.bfloat16)  # noqa: E731
    freq = ref.frequencies(64).cuda()
    assert lib.rotary(bf(0, 4, 64), bf(0, 2, 64), freq)[0].shape == (0, 4, 64)
    assert lib.rotary(bf(2, 4, 0, 64), None, freq)[0].shape == (2, 4, 0, 64)
    pool, sc = e(5, 2, 16, 64, dtype=torch.uint8), e(5, 2, dtype=torch.uint8)
    assert lib.append_paged(bf(0, 2, 64), bf(0, 2, 64), e(0), pool, pool, sc, sc, q=bf(0, 4, 64)).shape == (0, 4, 64)
    assert lib.gather_paged(pool, pool, e(0, 3), e(0), 16, sc, sc)[0].shape == (0, 2, 16, 64)
    o, lse = lib.decode_paged_block_scaled(bf(0, 4, 64), pool, pool, sc, sc, e(0, 3), e(0))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    o, lse = lib.prefill_paged_block_scaled(bf(0, 4, 64), pool, pool, sc, sc, e(1, 3), _i32([0]).cuda(),
                                            cu_seqlens_q=_i32([0, 0]).cuda(), max_seqlen_q=0)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)


@gpu
@pytest.mark.parametrize("chunk", [2, 600])
def test_rows_behind_the_last_sequence_are_left_alone(lib, chunk):
    c = _decode_case([700, 650], 8, 2, 128, 42)
    dev = [c[n].cuda() for n in ("kc", "vc", "ks", "vs", "table")]
    q = torch.randn(2 * chunk + 5, 8, 128, generator=_gen(1)).to(torch.bfloat16).cuda()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, q.shape[0]), 7.0, dtype=torch.float32, device="cuda")
    lib.prefill_paged_block_scaled(q, *dev, _i32(c["lens"]).cuda(), out=out, lse=lse,
                                   cu_seqlens_q=_i32([0, chunk, 2 * chunk]).cuda(), max_seqlen_q=chunk)
    assert (out[2 * chunk:] == 7.0).all() and (lse[:, 2 * chunk:] == 7.0).all()
    assert (out[: 2 * chunk] != 7.0).any(-1).all() and torch.isfinite(lse).all()


@gpu
@pytest.mark.parametrize("chunk,context", [(3, 900), (200, 2000)])
def test_prefill_block_scaled_in_a_graph_and_on_two_streams(lib, chunk, context):
    """Captured and replayed, and two calls at once on two streams: the bits of a call by itself."""
    cases = []
    for seed in (51, 52):
        c = _decode_case([chunk + context, chunk + context // 3], 8, 2, 128, seed)
        q = torch.randn(2, 8, chunk, 128, generator=_gen(seed)).to(torch.bfloat16).cuda()
        dev = [c[n].cuda() for n in ("kc", "vc", "ks", "vs", "table")]
        cases.append(lambda q=q, dev=dev, lens=_i32(c["lens"]).cuda(): lib.prefill_paged_block_scaled(q, *dev, lens))
    want = [f() for f in cases]
    torch.cuda.synchronize()
    graphs = []
    for f in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f()
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        both = []
        for f, s in zip(cases, streams):
            with torch.cuda.stream(s):
                both.append(f())
        torch.cuda.synchronize()
        for w, (_, o), e in zip(want, graphs, both):
            assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1]) and torch.equal(w[0], e[0]) and torch.equal(w[1], e[1])


@gpu
def test_decode_block_scaled_strided_views_are_refused(lib):
    c = _decode_case([40, 40], 4, 2, 64, 60)
    dev = [c[n].cuda() for n in ("kc", "vc", "ks", "vs", "table")]
    lens, q = _i32(c["lens"]).cuda(), c["q"].cuda()
    wide = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    for args in ((wide[:, :, :64], *dev, lens), (q, dev[0].transpose(0, 1), *dev[1:], lens),
                 (q, dev[0], dev[1], dev[2].int(), *dev[3:], lens), (q, *dev, lens.long()), (q.float(), *dev, lens),
                 (q, *dev[:4], dev[4][:1], lens)):
        with pytest.raises(ValueError):
            lib.decode_paged_block_scaled(*args)


@gpu
def test_error_words_of_another_type_are_refused(lib):
    c = _decode_case([40, 40], 4, 2, 64, 61)
    dev = [c[n].cuda() for n in ("kc", "vc", "ks", "vs", "table")]
    lens, q = _i32(c["lens"]).cuda(), c["q"].cuda()
    rows, slots = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda"), _i32([-1, -1]).cuda()
    one = _i32([0]).cuda()
    for flags in (torch.zeros(8, dtype=torch.uint8, device="cuda")[1:], torch.zeros(0, dtype=torch.int32, device="cuda")):
        for call in (lambda: lib.decode_paged_block_scaled(q, *dev, lens, error_flags=flags),
                     lambda: lib.prefill_paged_block_scaled(q[:, :, None], *dev, lens, error_flags=flags),
                     lambda: lib.append_paged(rows, rows, slots, *dev[:4], error_flags=flags),
                     lambda: lib.gather_paged(dev[0], dev[1], dev[4], lens, 40, dev[2], dev[3], error_flags=flags),
                     lambda: lib.plan_paged_step(lens.clone(), slots, dev[4], slots, one, 0, 9, error_flags=flags)):
            with pytest.raises(ValueError):
                call()


@gpu
def test_debug_build_finds_nothing(lib):
    """The bounds-checking build over decode (one and several clusters) and both prefill paths: no flag."""
    code = """
import sys; sys.path.insert(0, %r)
import torch
from attention_tiled_exact_b200 import binding as lib
from tests import test_paged_cache as t
assert lib.debug_bounds_enabled()
for splits in (0, 1, 16):
    assert t._decode_run(lib, t._decode_case([1, 0, 2500, 300], 9, 3, 128, 1), num_splits=splits)[2] == 0
c = t._decode_case([900, 640], 16, 2, 128, 2)
dev = [c[n].cuda() for n in ("kc", "vc", "ks", "vs", "table")]
for rows in (3, 600):
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 16, rows, 128, dtype=torch.bfloat16, device="cuda")
    lib.prefill_paged_block_scaled(q, *dev, t._i32(c["lens"]).cuda(), error_flags=flags)
    assert int(flags.item()) == 0
print("clean")
""" % ROOT
    env = dict(os.environ, ATTN_B200_DEBUG_BOUNDS="1")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600, env=env, cwd=ROOT)
    assert r.returncode == 0 and "clean" in r.stdout, r.stdout + r.stderr


# ---------------------------------------------------------------------------- together


@gpu
@pytest.mark.parametrize("fp8", [True, False])
def test_serving_steps_together(lib, fp8):
    """A prompt step and then decode steps in one captured graph, against attention in 64 bits over what the
    gather reads back, and the gather against the rows that were appended."""
    g = _gen(31)
    B, Hq, Hk, D, steps = 5, 8, 2, 128, 20
    freq = ref.frequencies(D).cuda()
    prompts = [17, 1, 0, 33, 64]
    width = 8
    nb = B * width + 1
    dtype = torch.uint8 if fp8 else torch.bfloat16
    kc, vc = (torch.full((nb, Hk, 16, D), 0x7F if fp8 else math.nan, dtype=dtype, device="cuda") for _ in range(2))
    ks, vs = (torch.full((nb, Hk), 255, dtype=torch.uint8, device="cuda") if fp8 else None for _ in range(2))
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(nb, generator=g).to(torch.int32).cuda()
    used, lens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = [[] for _ in range(B)]  # every sequence's appended (k, v) in order

    def keep(qkv, new):
        at = 0
        for b, n in enumerate(new):
            rows[b].append(qkv[at:at + n, Hq:].cpu())
            at += n

    # the prompts, in rows padded to a multiple of 64
    total = -(-sum(prompts) // 64) * 64
    qkv = torch.randn(total, Hq + 2 * Hk, D, generator=g).to(torch.bfloat16).cuda()
    keep(qkv, prompts)
    _, cu, pos, slots, _ = lib.plan_paged_step(lens, _i32(prompts).cuda(), table, free, used, total, nb, seq_lens_out=lens,
                                               num_used_out=used, error_flags=flags)
    q = lib.append_paged(qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], slots, kc, vc, ks, vs, q=qkv[:, :Hq], inv_freq=freq,
                         positions=pos, error_flags=flags)
    if fp8:
        o, lse = lib.prefill_paged_block_scaled(q, kc, vc, ks, vs, table, lens, cu_seqlens_q=cu, max_seqlen_q=64,
                                                max_seqlen_k=64, error_flags=flags)
    else:
        o, lse = lib.prefill_paged(q, kc, vc, table, lens, cu_seqlens_q=cu, max_seqlen_q=64, error_flags=flags)

    def check(q, o, new, pos):
        n_now = lens.tolist()
        dk, dv = (t.cpu().double() for t in lib.gather_paged(kc, vc, table, lens, width * 16, ks, vs))
        at = 0
        for b, n in enumerate(new):
            kr = torch.cat([r[:, :Hk] for r in rows[b]])[: n_now[b]] if rows[b] else None
            if n_now[b]:
                turned, size = ref.rotate_ref(kr.double(), torch.arange(n_now[b])[:, None], freq.cpu())
                top = turned.abs().amax()  # a block's scale is at most 2^-7.8 of its largest element
                step = 2.0 ** -4 if fp8 else BF16
                _within(dk[b, :, : n_now[b]].transpose(0, 1), turned, turned.abs() * step * 1.001 + size * ref.TURN_REL +
                        (top * 2.0 ** -16 if fp8 else 0), "keys")
            k, v = dk[b, :, : n_now[b]], dv[b, :, : n_now[b]]
            for i in range(n):
                limit = n_now[b] - n + i + 1
                qs = q[at + i].double().cpu().reshape(Hk, Hq // Hk, D)
                want, _, pv, size, _ = ref.attend_ref(qs, k, v, D ** -0.5, torch.full((Hq // Hk,), limit))
                tol = pv * (2.0 ** -8 + 2.0 ** -10) + want.abs() * BF16 + 2.0 ** -16 * (1 + size)[..., None] * pv + 2.0 ** -20
                _within(o[at + i].reshape(Hk, Hq // Hk, D), want, tol, f"step O {b}")
            at += n

    check(q, o, prompts, pos)
    # decode: one token each, the whole step in a graph over static buffers
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    x = torch.zeros(B, Hq + 2 * Hk, D, dtype=torch.bfloat16, device="cuda")
    out = {}

    def step():
        _, _, p, s, _ = lib.plan_paged_step(lens, one, table, free, used, B, nb, seq_lens_out=lens, num_used_out=used,
                                            error_flags=flags)
        out["q"] = lib.append_paged(x[:, Hq:Hq + Hk], x[:, Hq + Hk:], s, kc, vc, ks, vs, q=x[:, :Hq], inv_freq=freq,
                                    positions=p, error_flags=flags)
        if fp8:
            out["o"], out["lse"] = lib.decode_paged_block_scaled(out["q"], kc, vc, ks, vs, table, lens, num_splits=2,
                                                                 error_flags=flags)
        else:
            out["o"], out["lse"] = lib.decode_paged(out["q"], kc, vc, table, lens, num_splits=2, error_flags=flags)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # every kernel's set-up, on copies of nothing: the state is put back below
        saved = [t.clone() for t in (lens, table, used, kc, vc) + ((ks, vs) if fp8 else ())]
        step()
        for t, s in zip((lens, table, used, kc, vc) + ((ks, vs) if fp8 else ()), saved):
            t.copy_(s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        fresh = torch.randn(B, Hq + 2 * Hk, D, generator=g).to(torch.bfloat16)
        x.copy_(fresh.cuda())
        graph.replay()
        keep(fresh, [1] * B)
        if i % 5 == 4:
            check(out["q"], out["o"], [1] * B, None)
    assert int(flags.item()) == 0
    assert lens.tolist() == [p + steps for p in prompts]


# ---------------------------------------------------------------------------- refusals (no GPU)


FAKE = 1 << 20  # 16-byte aligned, never dereferenced: validation fails or no device is found first


def test_new_struct_layouts_match_the_header(lib):
    structs = {"attn_rotary_params": lib.RotaryParams, "attn_plan_params": lib.PlanParams,
               "attn_append_params": lib.AppendParams, "attn_gather_params": lib.GatherParams}
    body = ['#include <stdio.h>', '#include <stddef.h>', '#include "attn.h"', "int main(void){"]
    for name, s in structs.items():
        body.append(f'printf("{name} %zu\\n", sizeof({name}));')
        body += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in s._fields_]
    body.append("return 0;}")
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "probe.c"), os.path.join(d, "probe")
        open(c, "w").write("\n".join(body))
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = dict(line.split() for line in subprocess.run([exe], capture_output=True, text=True).stdout.splitlines())
    for name, s in structs.items():
        assert int(got[name]) == ctypes.sizeof(s)
        for f, _ in s._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(s, f).offset, (name, f)


def test_packed_parameters_are_the_structs(lib):
    """The bytes that the calls pass equal the ctypes mirror with the same fields."""
    for cls in (lib.PlanParams, lib.RotaryParams, lib.AppendParams, lib.GatherParams, lib.DecodeParams, lib.PrefillParams):
        args = [i + 0.5 if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(cls._fields_)]
        packed, mirror = lib._packer(cls)(*args), bytes(cls(*args))
        assert mirror.startswith(packed) and not any(mirror[len(packed):])


def _params(cls, **kw):
    p = cls()
    for name, typ in cls._fields_:
        if typ is ctypes.c_void_p:
            setattr(p, name, FAKE)
        elif name.endswith("_stride"):
            setattr(p, name, 1024)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _rotary(lib, **kw):
    base = dict(batch=2, num_q_heads=4, num_k_heads=2, seqlen=8, head_dim=128, rotary_dim=64, magnitude=1.0,
                q_out=2 * FAKE, k_out=2 * FAKE)
    return _params(lib.RotaryParams, **{**base, **kw})


@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 96, 2), ("rotary_dim", 24, 2), ("rotary_dim", 144, 1), ("rotary_dim", -16, 1), ("batch", -1, 1),
    ("seqlen", -1, 1), ("num_q_heads", 0, 1), ("num_k_heads", 0, 1), ("q", 0, 1), ("q_out", 0, 1), ("k_out", 0, 1),
    ("inv_freq", 0, 1), ("magnitude", math.nan, 1), ("in_dtype", 2, 1), ("out_dtype", 5, 1), ("q", FAKE + 8, 2),
    ("k_row_stride", 100, 2), ("qo_head_stride", 4, 2), ("seqlen", 0, 0), ("batch", 0, 0),
])
def test_rotary_refusals(lib, field, value, code):
    assert lib.LIB.attn_rotary(ctypes.byref(_rotary(lib, **{field: value})), None) == code


def test_rotary_refuses_unequal_views_in_place(lib):
    assert lib.LIB.attn_rotary(ctypes.byref(_rotary(lib, q_out=FAKE, qo_row_stride=2048)), None) == 1
    assert lib.LIB.attn_rotary(ctypes.byref(_rotary(lib, q_out=FAKE, out_dtype=1)), None) == 1
    assert lib.LIB.attn_rotary(None, None) == 1


@pytest.mark.parametrize("field,value,code", [
    ("batch", -1, 1), ("batch", 70000, 1), ("max_blocks_per_seq", 0, 1), ("num_blocks", 0, 1),
    ("num_blocks", 2 ** 27, 1), ("num_free", -1, 1), ("total_q", -1, 1), ("block_size", 32, 2), ("seq_lens", 0, 1),
    ("block_table", 0, 1), ("num_used", 0, 1), ("num_used_out", 0, 1), ("cu_seqlens_q", 0, 1), ("positions", 0, 1),
    ("slot_map", 0, 1), ("free_blocks", 0, 1), ("seq_lens_out", 0, 1), ("new_lens", 0, 1),
])
def test_plan_refusals(lib, field, value, code):
    p = _params(lib.PlanParams, batch=3, max_blocks_per_seq=4, num_blocks=9, num_free=2, total_q=3, block_size=16)
    setattr(p, field, value)
    assert lib.LIB.attn_plan_paged_step(ctypes.byref(p), None) == code


@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 32, 2), ("rotary_dim", 8, 2), ("total", -1, 1), ("num_kv_heads", 0, 1), ("num_q_heads", 0, 1),
    ("k", 0, 1), ("v_cache", 0, 1), ("k_scales", 0, 1), ("slot_map", 0, 1), ("positions", 0, 1), ("q_out", 0, 1),
    ("kv_dtype", 1, 1), ("kv_dtype", 9, 1), ("block_size", 8, 2), ("num_blocks", 2 ** 28, 1), ("v", FAKE + 2, 2),
    ("k_cache", FAKE + 8, 2), ("v_row_stride", 12, 2), ("qo_row_stride", 512, 1), ("total", 0, 0),
])
def test_append_refusals(lib, field, value, code):
    p = _params(lib.AppendParams, total=5, num_q_heads=4, num_kv_heads=2, head_dim=64, num_blocks=9, block_size=16,
                rotary_dim=32, magnitude=1.0, kv_dtype=2)
    setattr(p, field, value)
    assert lib.LIB.attn_append_paged(ctypes.byref(p), None) == code


@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 80, 2), ("batch", -1, 1), ("width", -1, 1), ("num_blocks", 0, 1), ("block_size", 4, 2),
    ("kv_dtype", 1, 1), ("v_scales", 0, 1), ("k_out", FAKE + 4, 2), ("block_table", 0, 1), ("max_blocks_per_seq", 0, 1),
    ("width", 0, 0), ("batch", 0, 0),
])
def test_gather_refusals(lib, field, value, code):
    p = _params(lib.GatherParams, batch=2, num_kv_heads=2, head_dim=64, width=40, num_blocks=9, block_size=16,
                max_blocks_per_seq=3, kv_dtype=2)
    setattr(p, field, value)
    assert lib.LIB.attn_gather_paged(ctypes.byref(p), None) == code


def _decode_params(lib, **kw):
    base = dict(batch=4, num_q_heads=12, num_kv_heads=4, head_dim=64, block_size=16, max_blocks_per_seq=100,
                num_blocks=500, scale=0.1, kv_dtype=2)
    return _params(lib.DecodeParams, **{**base, **kw})


@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 96, 2), ("num_q_heads", 10, 2), ("num_q_heads", 68, 2), ("num_kv_heads", 0, 1), ("block_size", 8, 2),
    ("scale", 0.0, 1), ("kv_dtype", 0, 1), ("o_dtype", 2, 1), ("q", 0, 1), ("o", FAKE + 4, 2), ("num_splits", -1, 1),
    ("max_blocks_per_seq", 0, 1), ("num_blocks", 2 ** 27, 1), ("batch", 70000, 1), ("head_dim", 128, 0),
])
def test_decode_block_scaled_refusals(lib, field, value, code):
    need = ctypes.c_size_t(0)
    p = _decode_params(lib, **{field: value})
    f = lib.LIB.attn_decode_paged_block_scaled
    assert f(ctypes.byref(p), FAKE, FAKE, None, 0, ctypes.byref(need), None) == code


def test_block_scaled_workspaces(lib):
    f = lib.LIB.attn_decode_paged_block_scaled
    need, need2 = ctypes.c_size_t(0), ctypes.c_size_t(0)
    p = _decode_params(lib, num_splits=16, max_blocks_per_seq=400)
    assert f(ctypes.byref(p), FAKE, FAKE, None, 0, ctypes.byref(need), None) == 0
    assert need.value >= 2 * 48 * 65 * 4 and need.value % 256 == 0
    assert f(ctypes.byref(p), FAKE, FAKE, FAKE, need.value - 256, ctypes.byref(need2), None) == lib.ATTN_ERR_WORKSPACE
    assert f(ctypes.byref(p), FAKE, FAKE, FAKE + 16, need.value, None, None) == lib.ATTN_ERR_UNSUPPORTED
    assert f(ctypes.byref(p), None, FAKE, None, 0, ctypes.byref(need), None) == lib.ATTN_ERR_INVALID_ARG
    p1 = _decode_params(lib, num_splits=1)
    assert f(ctypes.byref(p1), FAKE, FAKE, None, 0, ctypes.byref(need), None) == 0 and need.value == 0
    g = lib.LIB.attn_prefill_paged_block_scaled
    q = _params(lib.PrefillParams, batch=2, num_q_heads=4, num_kv_heads=2, head_dim=64, seqlen_q=8, seqlen_k=100,
                scale=0.1, k=0, v=0, max_blocks_per_seq=10, num_blocks=30, block_size=16, cu_seqlens_q=0)
    assert g(ctypes.byref(q), FAKE, FAKE, None, 0, ctypes.byref(need), None) == 0 and need.value % 256 == 0
    assert g(ctypes.byref(q), FAKE, None, None, 0, ctypes.byref(need), None) == lib.ATTN_ERR_INVALID_ARG
    if need.value:
        assert g(ctypes.byref(q), FAKE, FAKE, FAKE, need.value - 256, None, None) == lib.ATTN_ERR_WORKSPACE
    q.k_cache = 0
    q.v_cache = 0
    q.k = q.v = FAKE
    assert g(ctypes.byref(q), FAKE, FAKE, None, 0, ctypes.byref(need), None) == lib.ATTN_ERR_INVALID_ARG
    q.k = q.v = 0
    q.k_cache = q.v_cache = FAKE
    q.num_blocks = 2 ** 27
    assert g(ctypes.byref(q), FAKE, FAKE, None, 0, ctypes.byref(need), None) == lib.ATTN_ERR_INVALID_ARG


def test_python_checks_refuse_cpu_tensors_and_wrong_types(lib):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        lib.plan_paged_step(i(2), i(2), i(2, 3), i(4), i(1), 2, 9)
    with pytest.raises(ValueError):
        lib.rotary(torch.zeros(4, 2, 64), None, torch.zeros(32, dtype=torch.float64))
    z = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        lib.gather_paged(z, z, i(1, 2), i(1), 16)
    with pytest.raises(ValueError):
        lib.append_paged(torch.zeros(1, 2, 64), torch.zeros(1, 2, 64), i(1), z, z)
