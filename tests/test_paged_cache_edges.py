"""What the operators of a serving step over a paged cache do at their edges: requests over
their limits, scales far apart, far positions, paths that only some sizes take, faults."""
import ctypes

import pytest
import torch

from tests import paged_cache_ref as ref
from tests.test_paged_cache import _gen, _i32

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
