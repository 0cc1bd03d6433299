"""The paged 8-bit cache on the GPU against plain references (q8_ref.py): block
bookkeeping and codes bit for bit, attention within a bound derived from its
arithmetic (q8_ref.attention_tol)."""
import math
import random

import numpy as np
import pytest
import torch

import graph_community_sparse_b200 as ckv
import oracle.ckv_oracle as O
import q8_ref as Q
from parity_util import check_neighbours

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def table_lists(cache):
    bs = cache.desc.blocks.block
    lens = cache.len.tolist()
    t = cache.table.tolist()
    n_free = int(cache.blocks.n_free)
    return Q.Blocks(lens, [r[: -(-n // bs)] for r, n in zip(t, lens)], cache.blocks.free_list.tolist()[:n_free], bs,
                    cache.desc.blocks.max_blocks)


def check_table(cache, ref):
    bs, width = ref.block, ref.max_blocks
    assert cache.len.tolist() == ref.len
    assert cache.table.tolist() == [r + [-1] * (width - len(r)) for r in ref.table]
    n = int(cache.blocks.n_free)
    assert n == len(ref.free)
    assert cache.blocks.free_list.tolist()[:n] == ref.free
    held = [x for r in ref.table for x in r] + ref.free
    assert sorted(held) == list(range(cache.desc.blocks.n_blocks))  # nothing lost, nothing twice


def plan(cache, ref, add, n_rows, stream=None):
    p = ckv.new_plan(cache, n_rows)
    p.slot.fill_(77)
    ckv.ckv_plan_blocks(cache, i32(add), p, stream)
    start, slot, granted, refused = ref.change(add, n_rows)
    assert p.start.tolist() == start
    assert p.granted.tolist() == granted
    assert p.slot.tolist() == slot
    err = ckv.ckv_get_device_error(cache, reset=True)
    assert err == (ckv.DEVERR_PLAN if refused else 0)
    check_table(cache, ref)
    return p, granted


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("B,block,n_blocks,max_blocks,big", [
    (1, 16, 5, 5, 90), (3, 16, 40, 9, 40), (5, 64, 30, 7, 300), (33, 32, 200, 12, 60), (700, 16, 900, 4, 30),
    (1500, 16, 2500, 3, 20), (2, 128, 700, 400, 40000)])
def test_plan_follows_the_reference(B, block, n_blocks, max_blocks, big):
    """Random growth and drops, refusals of each kind among them; the slot map spans one block and a cluster of them."""
    rng = random.Random(B * 1000 + block)
    cache = ckv.new_q8_cache(B, 1, 1, 64, n_blocks, block, max_blocks)
    ref = table_lists(cache)
    for step in range(12):
        add = [rng.choice([0, 1, 1, rng.randint(1, big), -1, -rng.randint(1, big), -10 ** 9 if rng.random() < 0.1 else 2])
               for _ in range(B)]
        rows = sum(max(a, 0) for a in add)
        plan(cache, ref, add, max(0, rows + rng.choice([0, 0, 5, -3])))


def test_plan_reuses_blocks_of_a_drop_and_returns_to_the_same_state():
    cache = ckv.new_q8_cache(4, 1, 1, 64, 20, 16, 8)
    ref = table_lists(cache)
    plan(cache, ref, [17, 16, 0, 40], 73)
    before = (cache.table.clone(), cache.blocks.free_list.clone(), cache.blocks.n_free.clone())
    plan(cache, ref, [20, 1, 33, 0], 54)
    plan(cache, ref, [-20, -1, -33, 0], 0)
    assert torch.equal(before[0], cache.table) and torch.equal(before[2], cache.blocks.n_free)
    assert torch.equal(before[1][: int(before[2])], cache.blocks.free_list[: int(before[2])])
    # a request's end and another's start in one call: the free list alone would not do
    plan(cache, ref, [0, 0, 128, 64], 192)
    assert int(cache.blocks.n_free) < 4
    plan(cache, ref, [100, 0, -128, 0], 100)


def test_plan_zero_rows_and_empty_changes():
    cache = ckv.new_q8_cache(3, 1, 1, 64, 4, 16, 4)
    ref = table_lists(cache)
    plan(cache, ref, [0, 0, 0], 0)
    plan(cache, ref, [-5, 0, -1], 0)
    plan(cache, ref, [0, 1, 0], 0)      # no row: refused
    plan(cache, ref, [16, 16, 32], 64)  # exactly all blocks
    plan(cache, ref, [1, 1, 1], 3)      # full: refused, one and all
    plan(cache, ref, [-1, 1, 1], 2)     # 15 of 16: no block comes back
    plan(cache, ref, [1, -16, 1], 2)    # one does


def test_plan_huge_requests_do_not_overflow():
    cache = ckv.new_q8_cache(4, 1, 1, 64, 4, 16, 4)
    ref = table_lists(cache)
    big = 2 ** 31 - 1
    p = ckv.new_plan(cache, 8)
    ckv.ckv_plan_blocks(cache, i32([5, big, big, 3]), p)
    # the rows of the huge requests push request 3's past the slot map
    assert p.granted.tolist() == [5, 0, 0, 0]
    assert p.start.tolist() == [0, 5, big, big, big]
    assert p.slot.tolist() == [int(cache.table[0, 0]) * 16 + i for i in range(5)] + [-1] * 3
    assert ckv.ckv_get_device_error(cache, reset=True) == ckv.DEVERR_PLAN
    ref.change([5, 0, 0, 0], 8)
    check_table(cache, ref)
    ckv.ckv_plan_blocks(cache, i32([-2 ** 31, 0, 0, 0]), p)
    assert cache.len.tolist() == [0, 0, 0, 0] and int(cache.blocks.n_free) == 4


def test_plan_bad_lengths_are_flagged_and_left():
    cache = ckv.new_q8_cache(3, 1, 1, 64, 8, 16, 4)
    cache.len.copy_(i32([-3, 1000, 0]))
    p = ckv.new_plan(cache, 10)
    ckv.ckv_plan_blocks(cache, i32([4, -2, 4]), p)
    assert p.granted.tolist() == [0, 0, 4] and cache.len.tolist() == [-3, 1000, 4]
    assert p.slot.tolist()[:4] == [-1] * 4 and min(p.slot.tolist()[4:8]) >= 0
    assert ckv.ckv_get_device_error(cache, reset=True) == ckv.DEVERR_BLOCK | ckv.DEVERR_PLAN


def test_plan_bad_lengths_with_many_rows():
    """The rows of a request whose length is bad get no slot, lengths next to 2^31 among them."""
    cache = ckv.new_q8_cache(4, 1, 1, 64, 400, 16, 400)
    lens = [2 ** 31 - 1, -(2 ** 31), 400 * 16 + 1, 0]
    cache.len.copy_(i32(lens))
    p = ckv.new_plan(cache, 12000)
    ckv.ckv_plan_blocks(cache, i32([3000, 2999, 7, 5000]), p)
    assert p.granted.tolist() == [0, 0, 0, 5000] and cache.len.tolist() == lens[:3] + [5000]
    slot = p.slot.tolist()
    assert slot[:6006] == [-1] * 6006 and slot[11006:] == [-1] * (12000 - 11006)
    table = cache.table[3].tolist()
    assert slot[6006:11006] == [table[i // 16] * 16 + i % 16 for i in range(5000)]
    assert ckv.ckv_get_device_error(cache, reset=True) == ckv.DEVERR_BLOCK | ckv.DEVERR_PLAN


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------

def rows_for(add, Hkv, d, dtype, gen, spread=True):
    """Rows whose sizes vary from token to token, ties to the codes' borders and zeros among them."""
    N = sum(max(a, 0) for a in add)
    x = torch.randn((N, Hkv, d), generator=gen)
    if spread:
        x *= torch.exp2(torch.randint(-6, 4, (N, Hkv, 1), generator=gen).float())
        if N:
            x[:: 3, :, 0] = x[:: 3].abs().amax(-1)          # the row's largest
            x[:: 3, :, 1] = x[:: 3, :, 0] / 2                # 63.5 steps of it
            x[1:: 5] = 0.0
    return x.to(dtype)


def split_rows(x, add):
    out, at = [], 0
    for a in add:
        out.append(x[at: at + max(a, 0)].float().numpy())
        at += max(a, 0)
    return out


def check_pool(cache, refs, blocks):
    """Codes of every filled position, scales of every block in use, and the rest untouched by name."""
    for t, s, ref in ((cache.k, cache.k_scale, refs[0]), (cache.v, cache.v_scale, refs[1])):
        got, sc = Q.code_values(t), s.cpu().numpy()
        for b, n in enumerate(blocks.len):
            for j, blk in enumerate(blocks.table[b]):
                m = min(n - j * blocks.block, blocks.block)
                np.testing.assert_array_equal(sc[blk].astype(np.float64), ref.scales[blk])
                np.testing.assert_array_equal(got[blk, :, :m], ref.codes[blk, :, :m])


def refs_of(cache):
    fmt = "int8" if cache.k.dtype == torch.int8 else "e4m3"
    bs = cache.desc.blocks.block
    return [Q.Pool(Q.code_values(t), s.cpu().numpy(), bs, fmt)
            for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hkv,d,block", [(1, 64, 16), (3, 64, 128), (2, 128, 32), (2, 128, 64), (1, 128, 128),
                                         (5, 128, 16), (2, 64, 64), (1, 64, 32)])
def test_append_and_read(fmt, dtype, Hkv, d, block):
    """Several rounds of ragged growth and roll-backs: codes and scales bit for bit, and the rows read back."""
    gen = torch.Generator().manual_seed(block * d + Hkv)
    rng = random.Random(block + d + Hkv)
    B, cap = 4, 9
    cache = ckv.new_q8_cache(B, Hkv, Hkv, d, B * cap, block, cap, fmt, dtype)
    blocks, refs = table_lists(cache), refs_of(cache)
    for step in range(7):
        add = [rng.choice([1, 1, 0, -rng.randint(1, block), rng.randint(1, 2 * block)]) for _ in range(B)]
        if step == 0:
            add = [block + 3, 1, 0, 2 * block]
        k, v = rows_for(add, Hkv, d, dtype, gen), rows_for(add, Hkv, d, dtype, gen)
        p, granted = plan(cache, blocks, add, k.shape[0])
        ckv.ckv_quant_append(cache, p, k.to(DEV), v.to(DEV))
        refused = [a if g == a else 0 for a, g in zip(add, granted)]
        for ref, x in zip(refs, (k, v)):
            ref.append(blocks, granted, split_rows(x, add))
        check_pool(cache, refs, blocks)
        assert refused is not None and ckv.ckv_get_device_error(cache) == 0
    # read back, whole and from odd places
    for first, R in ((None, max(blocks.len) + 3), (i32([5, 0, 1, block - 1]), block + 1), (i32([0] * B), 1)):
        ko = torch.full((B, Hkv, R, d), 9.0, dtype=dtype, device=DEV)
        vo = torch.full_like(ko, 9.0)
        ckv.ckv_q8_read(cache, ko, vo, first)
        at = [0] * B if first is None else first.tolist()
        for b in range(B):
            pos = [x for x in range(at[b], at[b] + R) if x < blocks.len[b]]
            for out, ref in ((ko, refs[0]), (vo, refs[1])):
                want = np.zeros((R, Hkv, d))
                want[: len(pos)] = ref.rows(blocks, b, pos)
                want = torch.from_numpy(want).to(torch.float32).to(dtype)  # code * scale, rounded once each
                assert torch.equal(out[b].cpu().transpose(0, 1), want)
    assert ckv.ckv_get_device_error(cache) == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_raises_the_scale_of_a_part_filled_block(fmt):
    """Token by token with growing magnitudes: each new row re-scales the older codes."""
    cache = ckv.new_q8_cache(1, 2, 2, 64, 4, 16, 2, fmt, torch.float32)
    blocks, refs = table_lists(cache), refs_of(cache)
    gen = torch.Generator().manual_seed(3)
    for i in range(20):
        k = torch.randn((1, 2, 64), generator=gen) * 1.7 ** i
        v = torch.randn((1, 2, 64), generator=gen) * 0.9 ** i
        p, g = plan(cache, blocks, [1], 1)
        ckv.ckv_quant_append(cache, p, k.to(DEV), v.to(DEV))
        for ref, x in zip(refs, (k, v)):
            ref.append(blocks, g, split_rows(x, [1]))
        check_pool(cache, refs, blocks)


@pytest.mark.parametrize("layout", ["padded", "cache", "packed"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_row_layouts(layout, dtype):
    """Padded [B, T, Hkv, d], a view of a [B, Hkv, T, d] cache, packed rows with gaps: the same codes."""
    B, Hkv, d, T = 3, 2, 64, 40
    add = [40, 1, 17]
    gen = torch.Generator().manual_seed(5)
    full = torch.randn((2, B, T, Hkv, d), generator=gen).to(dtype)
    for b, a in enumerate(add):
        full[:, b, a:] = float("nan")  # padding: never read into a block
    cache = ckv.new_q8_cache(B, Hkv, Hkv, d, 12, 16, 4, "int8", dtype)
    blocks, refs = table_lists(cache), refs_of(cache)
    p, g = plan(cache, blocks, add, sum(add))
    if layout == "padded":
        rows = [x.to(DEV) for x in full]
    elif layout == "cache":
        rows = [x.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) for x in full]
    else:
        rows = []
        for x in full:
            wide = torch.full((sum(add), Hkv + 1, d + 8), float("nan"), dtype=dtype)
            wide[:, :Hkv, :d] = torch.cat([x[b, :a] for b, a in enumerate(add)])
            rows.append(wide.to(DEV)[:, :Hkv, :d])
    ckv.ckv_quant_append(cache, p, *rows)
    for ref, x in zip(refs, full):
        ref.append(blocks, g, [x[b, :a].float().numpy() for b, a in enumerate(add)])
    check_pool(cache, refs, blocks)
    assert ckv.ckv_get_device_error(cache) == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_extreme_values(fmt):
    """Zeros, magnitudes near the ends of fp32's range and subnormals keep finite codes and scales; a value that is
    not finite makes its own block's scale NaN and no other's."""
    cache = ckv.new_q8_cache(1, 1, 1, 64, 8, 16, 8, fmt, torch.float32)
    blocks, refs = table_lists(cache), refs_of(cache)
    x = torch.randn((96, 1, 64), generator=torch.Generator().manual_seed(1))
    x[:16] = 0.0
    x[16:32] *= 1e37
    x[32:48] *= 1e-42
    x[48:64] *= 2.0 ** -99
    x[64:80] = x[64:80].clamp(-1, 1) * 3.3895e38
    p, g = plan(cache, blocks, [96], 96)
    ckv.ckv_quant_append(cache, p, x.to(DEV), x.to(DEV))
    for ref in refs:
        ref.append(blocks, g, [x.numpy()])
    check_pool(cache, refs, blocks)
    assert torch.isfinite(cache.k_scale).all()
    for bad in (float("inf"), float("-inf"), float("nan")):
        y = torch.ones((33, 1, 64))
        y[20, 0, 7] = bad
        c2 = ckv.new_q8_cache(1, 1, 1, 64, 8, 16, 8, fmt, torch.float32)
        bl = table_lists(c2)
        p, g = plan(c2, bl, [33], 33)
        ckv.ckv_quant_append(c2, p, y.to(DEV), torch.ones((33, 1, 64), device=DEV))
        assert [math.isnan(float(c2.k_scale[b, 0])) for b in bl.table[0]] == [False, True, False]
        assert torch.isfinite(c2.v_scale).all()
        # a later row of that block does not hide it; a fresh use of the block clears it
        p, g = plan(c2, bl, [-8], 0)
        p, g = plan(c2, bl, [1], 1)
        one = torch.ones((1, 1, 64), device=DEV)
        ckv.ckv_quant_append(c2, p, one, one)
        assert math.isnan(float(c2.k_scale[bl.table[0][1], 0]))
        p, g = plan(c2, bl, [-26], 0)
        for _ in range(2):  # 16 tokens take one block; the second 16 the one that held the bad value
            p, g = plan(c2, bl, [16], 16)
            ckv.ckv_quant_append(c2, p, one.expand(16, 1, 64).contiguous(), one.expand(16, 1, 64).contiguous())
        assert torch.isfinite(c2.k_scale).all()


def test_append_leaves_the_rest_of_the_pool():
    cache = ckv.new_q8_cache(2, 2, 2, 64, 10, 16, 5)
    cache.k.copy_(torch.randint(-100, 100, cache.k.shape, dtype=torch.int8))
    cache.v.copy_(torch.randint(-100, 100, cache.v.shape, dtype=torch.int8))
    cache.k_scale.uniform_(1, 2)
    cache.v_scale.uniform_(1, 2)
    before = [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    blocks = table_lists(cache)
    p, g = plan(cache, blocks, [20, 5], 25)
    x = torch.randn((25, 2, 64), device=DEV).bfloat16()
    ckv.ckv_quant_append(cache, p, x, x)
    touched = torch.zeros((10, 16), dtype=torch.bool)
    for s in p.slot.tolist():
        touched[s // 16, s % 16] = True
    for now, old in ((cache.k, before[0]), (cache.v, before[1])):
        same = (now == old).cpu().all(-1).all(1)
        assert same[~touched].all()
    free = blocks.free
    assert torch.equal(cache.k_scale[free], before[2][free]) and torch.equal(cache.v_scale[free], before[3][free])


def test_append_bad_plans_are_flagged_and_skipped():
    """Slots out of range or off their row, growth beyond the length, rows or padding: nothing is written."""
    cache = ckv.new_q8_cache(1, 1, 1, 64, 4, 16, 4)
    cache.len.fill_(5)
    x = torch.ones((5, 1, 64), dtype=torch.bfloat16, device=DEV)

    def go(start, slot, granted, rows=x):
        p = ckv.Plan(i32(start), i32(slot), i32(granted))
        ckv.ckv_quant_append(cache, p, rows, rows)
        assert ckv.ckv_get_device_error(cache, reset=True) == ckv.DEVERR_BLOCK
        assert (cache.k == 0).all() and (cache.k_scale == 1).all()

    go([0, 5], [64, 65, 66, 67, 68], [5])             # past the pool
    go([0, 5], [-1] * 5, [5])
    go([0, 5], [1, 2, 3, 4, 5], [5])                  # row 1 for position 0
    go([0, 5], [0, 1, 2, 3, 4], [6])                  # more rows than the slot map has
    go([-2, 3], [0, 1, 2, 3, 4], [3])                 # before it
    cache.len.fill_(3)
    go([0, 5], [0, 1, 2, 3, 4], [5])                  # more than the length
    cache.len.fill_(65)
    go([0, 5], [0, 1, 2, 3, 4], [5])                  # a length past the table
    cache.len.fill_(5)
    go([0, 5], [0, 1, 2, 3, 4], [5], torch.ones((1, 3, 1, 64), dtype=torch.bfloat16, device=DEV))  # past the padding
    padded = torch.ones((1, 5, 1, 64), dtype=torch.bfloat16, device=DEV)
    go([3, 8], [0, 1, 2, 3, 4], [5], padded)          # slots past the slot map, whatever the rows' layout
    go([-1, 4], [0, 1, 2, 3, 4], [5], padded)


def test_read_bad_blocks_are_zeros():
    cache = ckv.new_q8_cache(2, 1, 1, 64, 4, 16, 4)
    cache.k.fill_(3)
    cache.v.fill_(3)
    cache.len.copy_(i32([20, 70]))
    cache.table.copy_(torch.tensor([[1, 9, -1, -1], [0, 2, 3, 1]], dtype=torch.int32))
    ko = torch.full((2, 1, 30, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    vo = torch.full_like(ko, 5.0)
    ckv.ckv_q8_read(cache, ko, vo, i32([0, -3]))
    assert (ko[0, 0, :16] == 3).all() and (ko[0, 0, 16:] == 0).all()  # block 9 does not exist
    assert (ko[1] == 0).all() and (vo[1] == 0).all()                  # a length past the table
    assert ckv.ckv_get_device_error(cache) == ckv.DEVERR_BLOCK


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def filled(lens, Hkv, Hq, d, block, fmt, dtype, seed, spread=1.0, spare=2):
    """A cache with random codes in blocks of random order; unused rows and blocks hold junk."""
    gen = torch.Generator().manual_seed(seed)
    nb = [-(-n // block) for n in lens]
    n_blocks = sum(nb) + spare
    cache = ckv.new_q8_cache(len(lens), Hkv, Hq, d, n_blocks, block, max(max(nb), 1) + 1, fmt, dtype)
    order = torch.randperm(n_blocks, generator=gen).tolist()
    at, rows = 0, []
    for n in nb:
        rows.append(order[at: at + n] + [-1] * (cache.desc.blocks.max_blocks - n))
        at += n
    cache.table.copy_(torch.tensor(rows, dtype=torch.int32))
    cache.len.copy_(i32(lens))
    cache.blocks.n_free.fill_(n_blocks - at)
    cache.blocks.free_list[: n_blocks - at] = i32(order[at:])
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        if fmt == "int8":
            c.copy_(torch.randint(-127, 128, c.shape, generator=gen, dtype=torch.int32).to(torch.int8))
        else:
            c.copy_((torch.randn(c.shape, generator=gen) * 90).clamp(-448, 448).to(torch.float8_e4m3fn))
        s.copy_(torch.exp2(spread * torch.randn(s.shape, generator=gen)) / (73 if fmt == "int8" else 90))
    # what no request holds must not matter
    for b, n in enumerate(lens):
        if n % block:
            last = rows[b][nb[b] - 1]
            cache.k.view(torch.uint8)[last, :, n % block:] = 127   # NaN in e4m3
            cache.v.view(torch.uint8)[last, :, n % block:] = 127
    for x in order[at:]:
        cache.k_scale[x] = float("nan")
        cache.v_scale[x] = float("inf")
    return cache


def check_out(cache, q, out, lists=None, group=True):
    """out against the reference on each head's positions (lists: [U] selected positions, else all)."""
    blocks = table_lists(cache)
    refs = refs_of(cache)
    B, Hq, d = q.shape
    Hkv = cache.desc.Hkv
    r = Hq // Hkv
    qn, on = q.double().cpu().numpy(), out.double().cpu().numpy()
    assert np.isfinite(on).all()
    worst = 0.0
    for b in range(B):
        n = blocks.len[b]
        k, v = (ref.rows(blocks, b, range(n)) for ref in refs)
        for h in range(Hq):
            g = h // r
            if lists is None:
                pos = np.arange(n)
            else:
                pos = np.asarray(lists[b * (Hkv if group else Hq) + (g if group else h)], dtype=np.int64)
            want, S = Q.attention(qn[b, h], k[pos, g], v[pos, g])
            tol = Q.attention_tol(S, len(pos), float(np.abs(v[pos, g]).max()) if len(pos) else 0.0)
            err = float(np.abs(on[b, h] - want).max())
            assert err <= tol, (b, h, len(pos), err, tol)
            worst = max(worst, err / tol if tol else 0.0)
    return worst


def workspace(cache, graph=None, sel=None):
    return ckv.new_workspace(ckv.ckv_q8_workspace_size(cache, graph, sel))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gq", [1, 2, 4, 8])
def test_dense_heads_and_types(fmt, dtype, d, gq):
    """Every head ratio, format and type, with lengths of 0, 1, whole and part-filled blocks and tiles."""
    lens = [0, 1, 15, 16, 17, 64, 100, 333, 0]
    cache = filled(lens, 2, 2 * gq, d, 32, fmt, dtype, seed=gq + d)
    q = torch.randn((len(lens), 2 * gq, d), device=DEV).to(dtype)
    out = torch.full(q.shape, float("nan"), device=DEV)
    ws = workspace(cache)
    ckv.ckv_dense_decode_q8(cache, q, out, ws)
    check_out(cache, q, out)
    assert (out[0] == 0).all() and (out[-1] == 0).all()
    first = out.clone()
    ckv.ckv_dense_decode_q8(cache, q, out, ws)  # the workspace is as it was; sums in a fixed order
    assert torch.equal(first, out)
    assert ckv.ckv_get_device_error(cache) == 0
    assert not ws[: 256 + 256].any()


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("lens", [[5000], [3, 4100, 129, 1, 640, 2500], [1] * 70, [257] * 40])
def test_dense_lengths_and_blocks(block, lens):
    """One request over many blocks of the grid, a ragged batch, many short ones."""
    cache = filled(lens, 3, 12, 128, block, "int8", torch.bfloat16, seed=len(lens))
    q = torch.randn((len(lens), 12, 128), device=DEV).bfloat16()
    out = torch.full(q.shape, float("nan"), device=DEV)
    ckv.ckv_dense_decode_q8(cache, q, out, workspace(cache))
    check_out(cache, q, out)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("gq", [4, 8])
def test_dense_scales_of_very_different_size(fmt, gq):
    """K scales that make the softmax sharp, V scales over 2^40: the tokens with weight decide, however large the others'
    values are."""
    lens = [700, 90]
    cache = filled(lens, 1, gq, 64, 16, fmt, torch.float32, seed=4, spread=1.5)
    cache.v_scale.copy_(torch.exp2(torch.randint(-20, 20, cache.v_scale.shape).float()))
    q = torch.randn((2, gq, 64), device=DEV) * 3
    q[0, 0] *= 1e-30
    q[0, 1] *= 1e-3
    q[1, 2] = 0.0
    q[1, 3, 5:] = 0.0
    out = torch.full(q.shape, float("nan"), device=DEV)
    ckv.ckv_dense_decode_q8(cache, q, out, workspace(cache))
    check_out(cache, q, out)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("gq", [4, 8])
def test_scales_of_zero(fmt, gq):
    """Blocks of all zeros kept with a scale of zero: scores and values of zero, in whole tiles, part-filled ones and
    lists."""
    lens = [100, 5, 32, 77]
    cache = filled(lens, 1, gq, 64, 16, fmt, torch.float32, seed=12)
    for b, blocks in enumerate(([0, 3], [0], [0, 1], [4])):
        for j in blocks:
            x = int(cache.table[b, j])
            cache.k_scale[x] = 0.0
            if b != 2 or j:
                cache.v_scale[x] = 0.0
    q = torch.randn((4, gq, 64), device=DEV)
    out = torch.full(q.shape, float("nan"), device=DEV)
    ckv.ckv_dense_decode_q8(cache, q, out, workspace(cache))
    check_out(cache, q, out)
    lists = [list(range(0, n, 2)) for n in lens]
    graph, sel = sparse_state(cache, lists, True, 0, 112)
    for nbr in (None, torch.empty((4, 8), dtype=torch.int32, device=DEV)):
        out.fill_(float("nan"))
        ckv.ckv_sparse_decode_q8(cache, q, graph, sel, out, nbr, workspace(cache, graph, sel))
        check_out(cache, q, out, lists)


def test_dense_one_token_far_in_a_large_pool():
    """Rows beyond 2^32 bytes of the pool."""
    Hkv, block, d = 8, 128, 128
    n_blocks = (2 ** 32 // (Hkv * block * d)) + 3
    cache = ckv.new_q8_cache(1, Hkv, Hkv, d, n_blocks, block, 2, "int8", torch.bfloat16)
    cache.table.copy_(torch.tensor([[n_blocks - 1, n_blocks - 2]], dtype=torch.int32))
    cache.len.fill_(200)
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c[n_blocks - 2:] = torch.randint(-127, 128, (2, Hkv, block, d), dtype=torch.int8, device=DEV)
        s.fill_(1 / 73)
    q = torch.randn((1, Hkv, d), device=DEV).bfloat16()
    out = torch.empty(q.shape, device=DEV)
    ckv.ckv_dense_decode_q8(cache, q, out, workspace(cache))
    ids = cache.table[0].long()
    for h in range(Hkv):
        k = cache.k[ids, h].reshape(-1, d)[:200].double().cpu().numpy() * float(cache.k_scale[0, 0])
        v = cache.v[ids, h].reshape(-1, d)[:200].double().cpu().numpy() * float(cache.v_scale[0, 0])
        want, S = Q.attention(q[0, h].double().cpu().numpy(), k, v)
        assert np.abs(out[0, h].double().cpu().numpy() - want).max() <= Q.attention_tol(S, 200, np.abs(v).max())


def test_dense_bad_blocks_and_lengths_are_skipped():
    lens = [100, 60, 40, 30]
    cache = filled(lens, 1, 4, 64, 16, "int8", torch.bfloat16, seed=9)
    q = torch.randn((4, 4, 64), device=DEV).bfloat16()
    good = torch.empty(q.shape, device=DEV)
    ckv.ckv_dense_decode_q8(cache, q, good, workspace(cache))
    cache.table[0, 2] = -1                       # positions 32..47 of request 0
    cache.table[1] = cache.desc.blocks.n_blocks  # all of request 1
    cache.len[2] = -7
    out = torch.full(q.shape, float("nan"), device=DEV)
    ckv.ckv_dense_decode_q8(cache, q, out, workspace(cache))
    assert ckv.ckv_get_device_error(cache, reset=True) == ckv.DEVERR_BLOCK
    assert (out[1] == 0).all() and (out[2] == 0).all()
    assert torch.equal(out[3], good[3])
    # request 0: the reference without those positions
    t = cache.table[0].tolist()
    pos = [p for p in range(100) if p // 16 != 2]
    k = np.stack([Q.code_values(cache.k[t[p // 16], 0, p % 16]) * float(cache.k_scale[t[p // 16], 0]) for p in pos])
    v = np.stack([Q.code_values(cache.v[t[p // 16], 0, p % 16]) * float(cache.v_scale[t[p // 16], 0]) for p in pos])
    for h in range(4):
        want, S = Q.attention(q[0, h].double().cpu().numpy(), k, v)
        assert np.abs(out[0, h].double().cpu().numpy() - want).max() <= Q.attention_tol(S, len(pos), np.abs(v).max())
    cache.len[2] = 10 ** 6
    ckv.ckv_dense_decode_q8(cache, q, out, workspace(cache))
    assert ckv.ckv_get_device_error(cache) == ckv.DEVERR_BLOCK and (out[2] == 0).all()


def test_dense_not_finite_values_reach_their_own_request_only():
    lens = [50, 50]
    cache = filled(lens, 2, 4, 64, 16, "int8", torch.float32, seed=2)
    cache.v_scale[cache.table[0, 1].long(), 0] = float("nan")
    q = torch.randn((2, 4, 64), device=DEV)
    out = torch.zeros(q.shape, device=DEV)
    ckv.ckv_dense_decode_q8(cache, q, out, workspace(cache))
    assert torch.isnan(out[0, :2]).all() and torch.isfinite(out[0, 2:]).all() and torch.isfinite(out[1]).all()
    q[1, 3, 0] = float("nan")
    q[1, 2, 0] = float("inf")
    ckv.ckv_dense_decode_q8(cache, q, out, workspace(cache))
    assert torch.isnan(out[1, 3]).all() and torch.isnan(out[1, 2]).all() and torch.isfinite(out[1, :2]).all()


# sparse -----------------------------------------------------------------

def sparse_state(cache, lists, group, S, T_cap, tok_cap=None):
    shape = ckv.q8_shape(cache, T_cap)
    graph = ckv.new_graph(shape, ckv.PER_GROUP if group else ckv.PER_HEAD, S, 4, 8)
    cap = tok_cap or max(max((len(x) for x in lists), default=0), S, 1)
    sel = ckv.new_selection(shape, graph, cap)
    sel.sel_tok.fill_(10 ** 6)  # behind the lists: never read
    for u, x in enumerate(lists):
        sel.sel_tok[u, : len(x)] = i32(x)
    sel.n_tok.copy_(i32([len(x) for x in lists]))
    return graph, sel


def random_lists(lens, G, sizes, S, rng):
    out = []
    for b, n in enumerate(lens):
        for g in range(G):
            m = min(n, sizes[(b * G + g) % len(sizes)])
            rest = rng.sample(range(min(S, n), n), max(0, m - S))
            out.append((list(range(min(S, n))) + rest) if m else [])
    return out


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,gq,group", [(64, 4, True), (128, 8, True), (128, 4, False), (128, 2, True), (64, 1, True),
                                        (128, 4, True), (64, 8, False)])
def test_sparse_lists(fmt, dtype, d, gq, group):
    """Lists of very different length (0, 1, odd, long) in a ragged batch, neighbours included."""
    lens = [0, 40, 700, 1300, 5]
    Hkv = 2
    rng = random.Random(d + gq)
    cache = filled(lens, Hkv, Hkv * gq, d, 64, fmt, dtype, seed=d + gq, spread=0.3)
    G = Hkv if group else Hkv * gq
    lists = random_lists(lens, G, [0, 1, 17, 333, 900, 64, 5], 3, rng)
    graph, sel = sparse_state(cache, lists, group, 3, 1344)
    q = torch.randn((len(lens), Hkv * gq, d), device=DEV).to(dtype)
    out = torch.full(q.shape, float("nan"), device=DEV)
    nbr = torch.full((graph.U, 8), -7, dtype=torch.int32, device=DEV)
    ws = workspace(cache, graph, sel)
    ckv.ckv_sparse_decode_q8(cache, q, graph, sel, out, nbr, ws)
    check_out(cache, q, out, lists, group)
    assert ckv.ckv_get_device_error(cache) == 0
    blocks, ref = table_lists(cache), refs_of(cache)[0]
    for u, pos in enumerate(lists):
        b, g = divmod(u, G)
        kv = g if group else g // gq
        heads = slice(g * gq, (g + 1) * gq) if group else slice(g, g + 1)
        K = np.zeros((max(lens), d))
        K[: lens[b]] = ref.rows(blocks, b, range(lens[b]))[:, kv]
        # a score is off by at most 14 * 2^-23 sum |q_i k_i| / sqrt(d), and so is the 8th
        qn = q[b, heads].double().cpu().numpy()
        S = float((np.abs(K[pos]) @ np.abs(qn).T).max() / math.sqrt(d)) if pos else 0.0
        if len(pos) == 0:
            assert nbr[u].tolist() == [-1] * 8
        else:
            check_neighbours(nbr[u].tolist(), qn, K, np.asarray(pos), 3, band=2 * 14 * 2.0 ** -23 * S)
    # without neighbours, by the other kernel
    out.fill_(float("nan"))
    ckv.ckv_sparse_decode_q8(cache, q, graph, sel, out, None, ws)
    check_out(cache, q, out, lists, group)
    first = out.clone()
    ckv.ckv_sparse_decode_q8(cache, q, graph, sel, out, None, ws)
    assert torch.equal(first, out) and not ws[: 256 + 32768].any()


@pytest.mark.parametrize("group", [True, False])
@pytest.mark.parametrize("B,n", [(40, 90), (3, 2500), (130, 20)])
def test_sparse_many_lists_and_long_ones(group, B, n):
    """More lists than blocks, lists that many blocks share, and a workspace that two caches use in turn."""
    Hkv, gq, d = 2, 4, 64
    lens = [n + (b * 7) % 31 for b in range(B)]
    cache = filled(lens, Hkv, Hkv * gq, d, 32, "int8", torch.bfloat16, seed=B)
    G = Hkv if group else Hkv * gq
    lists = random_lists(lens, G, [n, n // 2, 1, n - 3, 0, 16], 0, random.Random(B))
    graph, sel = sparse_state(cache, lists, group, 0, cache.desc.blocks.max_blocks * 32)
    q = torch.randn((B, Hkv * gq, d), device=DEV).bfloat16()
    ws = workspace(cache, graph, sel)
    other = filled([70, 900], 1, 8, 128, 16, "e4m3", torch.bfloat16, seed=1)
    q2 = torch.randn((2, 8, 128), device=DEV).bfloat16()
    out2 = torch.empty(q2.shape, device=DEV)
    if ws.numel() < ckv.ckv_q8_workspace_size(other):
        ws = workspace(other)
    for _ in range(2):
        out = torch.full(q.shape, float("nan"), device=DEV)
        ckv.ckv_sparse_decode_q8(cache, q, graph, sel, out, None, ws)
        ckv.ckv_dense_decode_q8(other, q2, out2, ws)
        ckv.ckv_dense_decode_q8(cache, q, torch.empty_like(out), ws)
    check_out(cache, q, out, lists, group)
    check_out(other, q2, out2)


def check_all_tokens(cache, q, out):
    """check_out's comparison over every token of an fp32 cache, on the GPU in float64."""
    n = cache.len.long()
    R = max(int(n.max()), 1)
    B, Hq, d = q.shape
    Hkv = cache.desc.Hkv
    k, v = (torch.empty((B, Hkv, R, d), device=DEV) for _ in range(2))
    ckv.ckv_q8_read(cache, k, v)
    k, v, qd = k.double().repeat_interleave(Hq // Hkv, 1), v.double().repeat_interleave(Hq // Hkv, 1), q.double()
    inside = (torch.arange(R, device=DEV) < n[:, None])[:, None]
    x = torch.einsum("bhd,bhtd->bht", qd, k) / math.sqrt(d)
    p = torch.softmax(x.masked_fill(~inside, -math.inf), -1).masked_fill(~inside, 0.0)  # an empty row: NaN, then 0
    want = torch.einsum("bht,bhtd->bhd", p, v)
    S = (torch.einsum("bhd,bhtd->bht", qd.abs(), k.abs()) / math.sqrt(d)).amax(-1)
    rel = 14 * 2.0 ** -23 * S + 3 * 2.0 ** -22 + 2.0 ** -23 * (n[:, None] / 128 + 308)  # Q.attention_tol, and the
    tol = 4 * rel * v.abs().amax((-1, -2))                                             # read rows' own rounding
    err = (out.double() - want).abs().amax(-1)
    assert bool((err <= tol).all()), float((err - tol).max())


def test_largest_batch():
    """8192 requests, the most a table may have: plan, append, dense and sparse attention."""
    B, gen = 8192, torch.Generator().manual_seed(3)
    cache = ckv.new_q8_cache(B, 1, 1, 64, 3 * B, 16, 3, "int8", torch.float32)
    ref = table_lists(cache)
    lens = torch.randint(0, 49, (B,), generator=gen).tolist()
    p, _ = plan(cache, ref, lens, sum(lens))
    k, v = torch.randn((2, sum(lens), 1, 64), generator=gen).to(DEV)
    ckv.ckv_quant_append(cache, p, k, v)
    plan(cache, ref, [-(n // 2) if n % 3 else -n for n in lens], 0)
    assert not all(ref.len) and max(ref.len) < 25
    q = torch.randn((B, 1, 64), generator=gen).to(DEV)
    out = torch.full(q.shape, float("nan"), device=DEV)
    graph, sel = sparse_state(cache, [[]] * B, True, 0, 48, tok_cap=48)
    sel.sel_tok.copy_(torch.arange(48, dtype=torch.int32, device=DEV).expand(B, 48))
    sel.n_tok.copy_(cache.len)
    ws = workspace(cache, graph, sel)
    ckv.ckv_dense_decode_q8(cache, q, out, ws)
    check_all_tokens(cache, q, out)
    nbr = torch.full((B, 8), -7, dtype=torch.int32, device=DEV)
    for n8 in (None, nbr):
        out.fill_(float("nan"))
        ckv.ckv_sparse_decode_q8(cache, q, graph, sel, out, n8, ws)
        check_all_tokens(cache, q, out)
    assert torch.equal((nbr >= 0).sum(1), cache.len.clamp(max=8))
    assert ckv.ckv_get_device_error(cache) == 0


@pytest.mark.parametrize("lens", [[65535], [65536], [2048 * 32 + 1, 7], [2047, 2049, 8191, 8192, 8193]])
def test_dense_lengths_where_the_least_piece_changes(lens):
    """Units of 64, 256 and 2048 tiles and their neighbours."""
    cache = filled(lens, 1, 2, 64, 64, "int8", torch.float32, seed=len(lens))
    q = torch.randn((len(lens), 2, 64), device=DEV)
    out = torch.full(q.shape, float("nan"), device=DEV)
    ws = workspace(cache)
    ckv.ckv_dense_decode_q8(cache, q, out, ws)
    check_all_tokens(cache, q, out)
    assert not ws[: 256 + 8192 * 4].any()


def test_sparse_all_tokens_equals_dense():
    lens = [300, 77]
    cache = filled(lens, 2, 8, 128, 32, "e4m3", torch.bfloat16, seed=1)
    lists = [random.Random(u).sample(range(lens[u // 2]), lens[u // 2]) for u in range(4)]
    graph, sel = sparse_state(cache, lists, True, 0, 320)
    q = torch.randn((2, 8, 128), device=DEV).bfloat16()
    a, b = torch.empty(q.shape, device=DEV), torch.empty(q.shape, device=DEV)
    ws = workspace(cache, graph, sel)
    ckv.ckv_sparse_decode_q8(cache, q, graph, sel, a, None, ws)
    ckv.ckv_dense_decode_q8(cache, q, b, ws)
    check_out(cache, q, a)
    check_out(cache, q, b)


def test_sparse_bad_entries_are_skipped():
    """Positions outside the request, blocks outside the pool, a list longer than its capacity."""
    lens = [200, 50]
    cache = filled(lens, 1, 4, 64, 16, "int8", torch.bfloat16, seed=6)
    good = list(range(0, 200, 3))
    bad = []
    for i, p in enumerate(good):
        bad += [p] + ([[-1, 200, 2 ** 31 - 1, -2 ** 31, 250][i % 5]] if i % 4 == 0 else [])
    graph, sel = sparse_state(cache, [bad, [60, 70, -5]], True, 0, 208, tok_cap=len(bad))
    q = torch.randn((2, 4, 64), device=DEV).bfloat16()
    out = torch.full(q.shape, float("nan"), device=DEV)
    nbr = torch.full((2, 8), -7, dtype=torch.int32, device=DEV)
    ws = workspace(cache, graph, sel)
    sel.n_tok[0] = len(bad) + 1000
    ckv.ckv_sparse_decode_q8(cache, q, graph, sel, out, nbr, ws)
    assert ckv.ckv_get_device_error(cache, reset=True) == ckv.DEVERR_BLOCK
    check_out(cache, q, out, [good, []])
    assert set(nbr[0].tolist()) <= set(good)
    assert nbr[1].tolist() == [-1] * 8  # a skipped entry is no neighbour
    # the same without neighbours (one launch)
    out.fill_(float("nan"))
    ckv.ckv_sparse_decode_q8(cache, q, graph, sel, out, None, ws)
    assert ckv.ckv_get_device_error(cache, reset=True) == ckv.DEVERR_BLOCK
    check_out(cache, q, out, [good, []])


@pytest.mark.parametrize("bad", [-1, 14 * 16 + 1, 2 ** 31 - 1])
@pytest.mark.parametrize("neighbours", [False, True])
def test_sparse_bad_length_skips_every_entry(bad, neighbours):
    cache = filled([200, 50], 1, 4, 64, 16, "int8", torch.bfloat16, seed=7)
    graph, sel = sparse_state(cache, [list(range(0, 200, 2)), list(range(50))], True, 0, 13 * 16, tok_cap=128)
    assert cache.desc.blocks.max_blocks == 14
    q = torch.randn((2, 4, 64), device=DEV).bfloat16()
    out = torch.full(q.shape, float("nan"), device=DEV)
    nbr = torch.full((2, 8), -7, dtype=torch.int32, device=DEV) if neighbours else None
    cache.len[0] = bad
    ckv.ckv_sparse_decode_q8(cache, q, graph, sel, out, nbr, workspace(cache, graph, sel))
    assert ckv.ckv_get_device_error(cache, reset=True) == ckv.DEVERR_BLOCK
    cache.len[0] = 200
    check_out(cache, q, out, [[], list(range(50))])
    if neighbours:
        assert nbr[0].tolist() == [-1] * 8 and min(nbr[1].tolist()) >= 0


def test_sparse_joins_communities_like_the_wide_cache():
    """Selection, attention and update over an 8-bit cache whose values a 16-bit one can hold exactly: the same
    neighbours, communities and centres as the framework's calls over that one."""
    B, Hkv, Hq, d, T, S, C = 2, 2, 8, 64, 500, 4, 12
    for group in (True, False):
        cache = ckv.new_q8_cache(B, Hkv, Hq, d, 80, 16, 40, "int8", torch.bfloat16)
        G = Hkv if group else Hq
        gen = torch.Generator().manual_seed(11)
        # integers up to 127 with a 127 in every block: scale 1, codes exact
        rows = torch.randint(-20, 21, (2, B, T, Hkv, d), generator=gen).float()
        rows[:, :, ::8, :, 0] = 127
        K, V = (x.bfloat16().to(DEV) for x in rows)
        p = ckv.new_plan(cache, B * T)
        ckv.ckv_plan_blocks(cache, i32([T] * B), p)
        ckv.ckv_quant_append(cache, p, K, V)
        used = cache.table[:, : -(-T // 16)].long().flatten()
        assert (cache.k_scale[used] == 1).all() and (cache.v_scale[used] == 1).all()
        ko, vo = (torch.zeros((B, Hkv, 512, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        ckv.ckv_q8_read(cache, ko, vo)
        assert torch.equal(ko[:, :, :T], K.transpose(1, 2)) and (ko[:, :, T:] == 0).all()
        wide = ckv.cache_desc(ko, vo, Hq)
        shape = ckv.q8_shape(cache, 512)
        mode = ckv.PER_GROUP if group else ckv.PER_HEAD
        graphs, sels, outs = [], [], []
        labels = torch.randint(0, C, (B * G, T), generator=gen, dtype=torch.int32).to(DEV)
        labels[:, :S] = -1
        q = (torch.randn((B, Hq, d), generator=gen) / 16).bfloat16().to(DEV)
        kn, vn = (torch.randint(-20, 21, (B, Hkv, d), generator=gen).bfloat16().to(DEV) for _ in range(2))
        for which in range(2):
            graph = ckv.new_graph(shape, mode, S, C, 8)
            sel = ckv.new_selection(shape, graph, 512)
            ws = ckv.new_workspace(ckv.ckv_workspace_size(wide, graph, sel))
            ckv.ckv_build_centroids(wide, labels, T, graph, ws)
            ckv.ckv_score_select(wide if which == 0 else shape, graph, q, 150, sel, ws)
            out = torch.empty((B, Hq, d), device=DEV)
            nbr = torch.empty((B * G, 8), dtype=torch.int32, device=DEV)
            asg = torch.empty((B * G,), dtype=torch.int32, device=DEV)
            if which == 0:
                ckv.ckv_sparse_decode_append(wide, q, graph, sel, out, nbr, T, kn, vn, asg, ws)
            else:
                ckv.ckv_sparse_decode_q8(cache, q, graph, sel, out, nbr, workspace(cache, graph, sel), kn, asg)
            assert int(graph.dev_err) == 0
            graphs.append(graph)
            outs.append((out, nbr, asg))
        assert torch.equal(outs[0][1], outs[1][1]) and torch.equal(outs[0][2], outs[1][2])
        # the wide attention keeps 16 bits of a weight (2^-16 of |v| <= 127) beside this one's bound
        assert float((outs[0][0] - outs[1][0]).abs().max()) <= 127 * 2.0 ** -15
        for f in ("comm_of", "cnt", "cent", "cent_q", "cent_qs", "tail_tok", "tail_comm", "tail_len"):
            assert torch.equal(getattr(graphs[0], f), getattr(graphs[1], f)), f


def test_sparse_join_at_each_requests_own_end():
    """Requests of different length: the new token joins at its own position; past T_cap it joins nothing."""
    lens = [30, 64, 47]
    cache = filled(lens, 1, 1, 64, 16, "int8", torch.float32, seed=8)
    shape = ckv.q8_shape(cache, 64)
    graph = ckv.new_graph(shape, ckv.PER_GROUP, 0, 2, 4)
    graph.comm_of.zero_()
    graph.cnt.fill_(1)
    graph.num_comm.fill_(2)
    sel = ckv.new_selection(shape, graph, 64)
    sel.sel_tok[:, :8] = torch.arange(8, dtype=torch.int32, device=DEV)
    sel.n_tok.fill_(8)
    q = torch.randn((3, 1, 64), device=DEV)
    out = torch.empty(q.shape, device=DEV)
    asg = torch.full((3,), -9, dtype=torch.int32, device=DEV)
    ckv.ckv_sparse_decode_q8(cache, q, graph, sel, out, None, workspace(cache, graph, sel),
                             torch.randn((3, 1, 64), device=DEV), asg)
    assert asg.tolist() == [0, -1, 0]
    assert graph.tail_tok[:, 0].tolist() == [30, 0, 47] and graph.tail_len.tolist() == [1, 0, 1]
    assert int(graph.dev_err) == ckv.DEVERR_INDEX


# ---------------------------------------------------------------------------
# streams, graphs, other uses
# ---------------------------------------------------------------------------

def test_run_of_them_on_a_stream_and_in_a_graph():
    """A decode step (slots, rows, dense attention) on a side stream, then captured and replayed: each replay continues
    from the state the one before left."""
    B, Hkv, Hq, d = 3, 2, 8, 64

    def fresh():
        cache = ckv.new_q8_cache(B, Hkv, Hq, d, 30, 16, 10, "int8", torch.bfloat16)
        gen = torch.Generator().manual_seed(0)
        x = torch.randn((2, 60, Hkv, d), generator=gen).bfloat16().to(DEV)
        p = ckv.new_plan(cache, 60)
        ckv.ckv_plan_blocks(cache, i32([31, 9, 20]), p)
        ckv.ckv_quant_append(cache, p, x[0], x[1])
        return cache

    add = i32([1, 1, 1])
    rows = torch.randn((2, B, Hkv, d), device=DEV).bfloat16()
    q = torch.randn((B, Hq, d), device=DEV).bfloat16()

    def step(cache, p, out, ws):
        ckv.ckv_plan_blocks(cache, add, p)
        ckv.ckv_quant_append(cache, p, rows[0], rows[1])
        ckv.ckv_dense_decode_q8(cache, q, out, ws)

    eager, captured = fresh(), fresh()
    outs = [torch.empty(q.shape, device=DEV) for _ in range(2)]
    plans = [ckv.new_plan(c, B) for c in (eager, captured)]
    wss = [workspace(c) for c in (eager, captured)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(captured, plans[1], outs[1], wss[1])
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(captured, plans[1], outs[1], wss[1])
    step(eager, plans[0], outs[0], wss[0])
    for _ in range(20):
        step(eager, plans[0], outs[0], wss[0])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
    assert torch.equal(eager.table, captured.table) and torch.equal(eager.k, captured.k)
    assert eager.len.tolist() == [52, 30, 41] == captured.len.tolist()
    check_out(captured, q, outs[1])
    assert ckv.ckv_get_device_error(captured) == 0


def test_the_debug_build_gives_the_same():
    lens = [100, 31]
    cache = filled(lens, 1, 4, 64, 16, "int8", torch.bfloat16, seed=3)
    q = torch.randn((2, 4, 64), device=DEV).bfloat16()
    a, b = torch.empty(q.shape, device=DEV), torch.empty(q.shape, device=DEV)
    ws = workspace(cache)
    ckv.ckv_dense_decode_q8(cache, q, a, ws)
    import ctypes
    dbg = ckv.load_debug_library()
    st = torch.cuda.current_stream().cuda_stream
    assert dbg.ckv_dense_decode_q8(ctypes.byref(cache.desc), q.data_ptr(), b.data_ptr(), ws.data_ptr(), ws.numel(), st) == 0
    torch.cuda.synchronize()
    assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# a layer's decode, as it is used
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("mode", ["group", "head"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_paged_layer_decodes_with_communities(mode, fmt):
    """Prompts written, communities built, then decode steps (select, attend with the join, grow, write) against the
    references: selections and joins of the oracle on the values that the cache holds."""
    from graph_community_sparse_b200.layer import PagedLayerState

    B, Hkv, Hq, d, T, S, C, steps = 2, 2, 4, 64, 300, 4, 10, 4
    gen = torch.Generator().manual_seed(17)
    cache = ckv.new_q8_cache(B, Hkv, Hq, d, 60, 16, 25, fmt, torch.float32)
    st = PagedLayerState(cache, mode, S, C, 8, T_cap=400)
    G = Hkv if mode == "group" else Hq
    mu = torch.randn((C, d), generator=gen)
    lab = torch.randint(0, C, (B, Hkv, T), generator=gen)
    K = (mu[lab] + 0.3 * torch.randn((B, Hkv, T, d), generator=gen)).to(DEV)
    V = torch.randn((B, Hkv, T, d), generator=gen).to(DEV)
    st.grow(i32([T, T]), B * T)
    st.write(K.transpose(1, 2), V.transpose(1, 2))
    labels = lab[:, :, None, :].expand(B, Hkv, G // Hkv, T).reshape(B * G, T).to(torch.int32).clone()
    labels[:, :S] = -1
    st.build(labels.to(DEV), T)
    blocks, refs = table_lists(cache), refs_of(cache)
    states = [O.GraphState(labels[u].numpy(), 400, S, C) for u in range(B * G)]
    # the keys that the centres average: the values held when the graphs were built, then the new tokens' own rows
    keys = np.zeros((B, Hkv, 400, d))
    for b in range(B):
        keys[b, :, :T] = refs[0].rows(blocks, b, range(T)).transpose(1, 0, 2)
    one = i32([1] * B)
    for step in range(steps):
        q = (0.5 * mu[torch.randint(0, C, (B, Hq), generator=gen)] + torch.randn((B, Hq, d), generator=gen)).to(DEV)
        kn, vn = torch.randn((2, B, Hkv, d), generator=gen).to(DEV)
        kn = kn + mu[0].to(DEV)
        st.select(q, 90)
        out = st.attend(q, kn).clone()
        lists = []
        for u in range(B * G):
            n = int(st.sel.n_tok[u])
            lists.append(st.sel.sel_tok[u, :n].tolist())
            b, g = divmod(u, G)
            kv = g if mode == "group" else g * Hkv // Hq
            heads = range(g * Hq // Hkv, (g + 1) * Hq // Hkv) if mode == "group" else [g]
            n_tok = blocks.len[b]
            members = states[u].members()
            cent, cnt = O.centroids(keys[b, kv], members)
            scores = O.community_scores(q[b, list(heads)].double().cpu().numpy(), cent, cnt)
            got = st.sel.sel_comm[u, : int(st.sel.n_sel[u])].tolist()
            want = O.select(scores, cnt, 90)
            # scores are fp32 sums of 64 products, a few units in size: 64 * 2^-24 * 8 < 1e-4
            cut = scores[want[-1]]
            assert all(abs(scores[c] - cut) < 1e-4 for c in set(got) ^ set(want)), (got, want)
            assert sorted(lists[-1]) == sorted(O.token_set(got, members, S).tolist())
            # the join: a candidate of the best score
            asg = int(st.assigned[u])
            cands = [int(states[u].comm_of[p]) for p in st.nbr8[u].tolist() if p >= 0]
            kk = kn[b, kv].double().cpu().numpy()
            best = max(float(kk @ cent[c]) for c in cands)
            assert asg in cands and best - float(kk @ cent[asg]) < 1e-4 * max(1.0, abs(best))
            states[u].comm_of[n_tok] = asg
            states[u].T = n_tok + 1
        check_out(cache, q, out, lists, mode == "group")
        p = st.grow(one, B)
        st.write(kn, vn)
        _, _, granted, _ = blocks.change([1] * B, B)
        for ref, x in zip(refs, (kn, vn)):
            ref.append(blocks, granted, split_rows(x.cpu(), [1] * B))
        check_table(cache, blocks)
        keys[:, :, T + step] = kn.double().cpu().numpy()
        assert p.granted.tolist() == [1] * B
    check_pool(cache, refs, blocks)
    check_out(cache, q, st.dense(q))
    assert cache.len.tolist() == [T + steps] * B
    assert ckv.ckv_get_device_error(cache) == 0 and int(st.graph.dev_err) == 0


def test_paged_layer_write_follows_grow():
    from graph_community_sparse_b200.layer import PagedLayerState

    st = PagedLayerState(ckv.new_q8_cache(1, 1, 1, 64, 4, 16, 4))
    with pytest.raises(RuntimeError):
        st.write(torch.zeros((1, 1, 64), dtype=torch.bfloat16, device=DEV), torch.zeros((1, 1, 64), dtype=torch.bfloat16, device=DEV))
    k, v = st.read(5)
    assert k.shape == (1, 1, 5, 64) and (k == 0).all() and (v == 0).all()


def test_paged_layer_on_another_stream():
    """Plans and rows that the layer makes belong to the stream of the call, busy or not current."""
    from graph_community_sparse_b200.layer import PagedLayerState

    st = PagedLayerState(ckv.new_q8_cache(2, 1, 1, 64, 700, 16, 350, "int8", torch.float32))
    one, other = i32([1, 1]), i32([5000, 0])
    rows = torch.randn((2, 5000, 1, 64), device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    junk = torch.zeros((1 << 27,), device=DEV)
    for _ in range(8):
        junk.add_(1)  # the current stream is behind: what it fills, it fills late
    small = st.grow(one, 2, s)
    st.write(rows[:, :1], rows[:, :1], s)
    large = st.grow(other, 5000, s.cuda_stream)
    st.write(rows[:, :], rows[:, :], s.cuda_stream)
    k, v = st.read(5001, stream=s)
    torch.cuda.synchronize()
    assert small.granted.tolist() == [1, 1] and large.granted.tolist() == [5000, 0]
    assert min(small.slot.tolist()) >= 0 and min(large.slot.tolist()) >= 0
    # half a step of a block's scale (largest magnitude / 127), and the roundings of the code's product; the
    # first row was re-scaled once, for another half
    step = float(rows.abs().max()) / 127
    assert (k[0, 0, 1:] - rows[0, :, 0]).abs().max() <= 0.501 * step
    assert (k[0, 0, 0] - rows[0, 0, 0]).abs().max() <= 1.002 * step
    assert torch.equal(k, v)
    assert st.grow(one, 2, s) is small and st.grow(other, 5000, s) is not large
