"""The operators of the paged 8-bit KV cache: what is measured, their plain
forms, and their definition in 64 bits.

The cache is a pool of blocks of ``block`` tokens.  A block holds, for each KV
head, ``block`` rows of d codes (int8 or e4m3) and one scale for K and one for
V.  A request's blocks are named by its row of the block table; positions
[0, len) of it are filled.

  plan    requests shrink or grow by a number of tokens each: blocks go back
          to the free list or are taken from it, and every new token gets its
          slot (block * block size + row)
  append  new K/V rows are quantised into their slots; what was written is
          read back in the rows' own type (as the prefill attention and the
          centroid build read it)
  dense   decode attention over all tokens of each request
  sparse  decode attention over each graph unit's list of selected positions
"""
import math

import torch

own = False

DEV = "cuda"
FLOOR = 2.0 ** -100  # the least magnitude a block's scale is made for


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a batch: 32 requests give back their speculative tokens and take new slots
        dict(name="plan decode", op="plan", B=32, block=64, lo=1000, hi=8000, add_lo=1, add_hi=8),
        # admission of prompts, 160K tokens over 48 requests
        dict(name="plan prompts", op="plan", B=48, block=16, lo=0, hi=300, add_lo=500, add_hi=6000),
        # a decode step's new rows, one per request
        dict(name="append token", op="append", B=8, Hkv=8, d=128, fmt="int8", dtype="bf16", block=64, lo=100, hi=4000,
             add_lo=1, add_hi=1),
        # ragged prompts that continue half-filled blocks, d = 64, fp32
        dict(name="append ragged", op="append", B=13, Hkv=3, d=64, fmt="int8", dtype="f32", block=32, lo=0, hi=200,
             add_lo=1, add_hi=900),
        # a whole 32K prompt
        dict(name="append prompt", op="append", B=1, Hkv=8, d=128, fmt="e4m3", dtype="bf16", block=64, lo=0, hi=0,
             add_lo=32768, add_hi=32768),
        # the smallest layer of this repository's workloads: 1 KV head, 1K tokens, fp32 queries
        dict(name="dense tiny", op="dense", B=1, Hq=4, Hkv=1, d=64, fmt="int8", dtype="f32", block=16, lo=1024, hi=1024),
        # one long request
        dict(name="dense one 32K", op="dense", B=1, Hq=32, Hkv=8, d=128, fmt="e4m3", dtype="bf16", block=64,
             lo=32768, hi=32768),
        # a ragged batch, from one token up
        dict(name="dense ragged", op="dense", B=33, Hq=32, Hkv=4, d=128, fmt="int8", dtype="bf16", block=32, lo=1, hi=9000),
        # a batch of long requests: the cache that fills the card
        dict(name="dense 128K", op="dense", B=8, Hq=32, Hkv=8, d=128, fmt="int8", dtype="bf16", block=64,
             lo=131072, hi=131072),
        # a small selection, d = 64, fp32 queries, one graph per group
        dict(name="sparse tiny", op="sparse", B=1, Hq=4, Hkv=1, d=64, fmt="int8", dtype="f32", block=16, T=1024, n=132,
             mode="group"),
        # one 32K request, one graph per KV group
        dict(name="sparse one 32K", op="sparse", B=1, Hq=32, Hkv=8, d=128, fmt="e4m3", dtype="bf16", block=64, T=32768,
             n=2052, mode="group"),
        # 128K tokens, one graph per query head
        dict(name="sparse 128K heads", op="sparse", B=8, Hq=32, Hkv=8, d=128, fmt="int8", dtype="bf16", block=64, T=131072,
             n=2052, mode="head"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "dense", "sparse"])
    block = rng.choice([16, 32, 64, 128])
    if op == "plan":
        lo = _log(rng, 1, 4000)
        add = _log(rng, 1, 3000)
        return dict(op=op, B=_log(rng, 1, 100), block=block, lo=lo, hi=lo + _log(rng, 1, 4000), add_lo=1 + add // 4, add_hi=add + 1)
    fmt, d = rng.choice(["int8", "e4m3"]), rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "append":
        B = _log(rng, 1, 40)
        add = _log(rng, 1, max(1, 32768 // B))
        lo = _log(rng, 1, 2000)
        return dict(op=op, B=B, Hkv=Hkv, d=d, fmt=fmt, dtype=dtype, block=block, lo=lo - 1, hi=lo + _log(rng, 1, 500),
                    add_lo=1 + add // 8, add_hi=add + 1)
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    B = _log(rng, 1, 40)
    if op == "dense":
        hi = _log(rng, 1, max(2, 400000 // B))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, fmt=fmt, dtype=dtype, block=block, lo=max(1, hi // rng.choice([1, 2, 50])), hi=hi)
    B = _log(rng, 1, 8)
    T = _log(rng, 64, 60000)
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, fmt=fmt, dtype=dtype, block=block, T=T, n=min(T, _log(rng, 8, 4200)),
                mode=rng.choice(["group", "head"]))


def _lengths(case):
    """The requests' lengths (before any growth) and their growth, from the case alone."""
    if "T" in case:
        return [case["T"]] * case["B"], [0] * case["B"]
    B, lo, hi = case["B"], case["lo"], case["hi"]
    n = [lo + (i * 2654435761 + 12345) % 4294967296 * (hi - lo + 1) // 4294967296 for i in range(B)]
    if "add_lo" not in case:
        return n, [0] * B
    a0, a1 = case["add_lo"], case["add_hi"]
    add = [a0 + (i * 2246822519 + 777) % 4294967296 * (a1 - a0 + 1) // 4294967296 for i in range(B)]
    return n, add


def _entries(case):
    """The lengths of the sparse lists, a little below the budget each."""
    U = case["B"] * (case["Hkv"] if case["mode"] == "group" else case["Hq"])
    return [case["n"] - u * 7919 % (case["n"] // 16 + 1) for u in range(U)]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def work(case):
    op = case["op"]
    if op == "plan":
        n, add = _lengths(case)
        bs = case["block"]
        moved = sum(-(-(x + a) // bs) - (-(-x // bs)) for x, a in zip(n, add))
        # per call: a request's growth and length read, length, start and grant written; a moved block's id read and
        # written in table and free list; the slots of the growing call
        return {"bytes": 2 * (case["B"] * 4 * 5 + moved * 8) + 4 * sum(add), "flops": 0}
    rows = 4 if case["dtype"] == "f32" else 2
    if op == "append":
        n, add = _lengths(case)
        N, bs = sum(add), case["block"]
        blocks = sum((x + a - 1) // bs - x // bs + 1 for x, a in zip(n, add))
        values = 2 * N * case["Hkv"] * case["d"]
        # the new rows in, their codes and the blocks' scales out, and the rows as read back out
        return {"bytes": values * (rows + 1 + rows) + blocks * case["Hkv"] * 8 + N * 4, "flops": 3 * values}
    Hq, Hkv, d, B = case["Hq"], case["Hkv"], case["d"], case["B"]
    if op == "dense":
        n, _ = _lengths(case)
        T = sum(n)
        blocks = sum(-(-x // case["block"]) for x in n)
        return {"bytes": T * Hkv * 2 * d + blocks * (4 + 8 * Hkv) + B * Hq * d * (rows + 4), "flops": 4 * T * Hq * d}
    G = Hkv if case["mode"] == "group" else Hq
    entries = sum(_entries(case))
    # heads of one group pick lists of their own; a row that several pick is read once
    distinct = case["T"] * (1 - (1 - entries / (B * G) / case["T"]) ** (G // Hkv)) * B * Hkv
    blocks = min(distinct, B * Hkv * -(-case["T"] // case["block"]))
    return {"bytes": distinct * 2 * d + entries * 4 + blocks * 8 + B * Hq * d * (rows + 4), "flops": 4 * entries * (Hq // G) * d}


# ---------------------------------------------------------------------------
# the inputs
# ---------------------------------------------------------------------------

def _quantise(x, fmt):
    """Blocks of rows [..., block, d] in fp32 as codes and scales (a scale per block)."""
    amax = x.abs().amax(dim=(-1, -2)).clamp_min(FLOOR)
    s = _scale(amax, fmt)
    y = x * (1.0 / s)[..., None, None]
    return (y.round().clamp(-127, 127).to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)), s


def _scale(amax, fmt):
    if fmt == "int8":
        return amax / torch.full_like(amax, 127.0)
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); the least power of two s with amax <= 448 s
    return ((e + 118 + (m > 0.875).to(e.dtype)) << 23).view(torch.float32)


def _pool(case, n_tokens, g, spare):
    """A pool whose requests hold n_tokens[b] tokens: clustered keys, normal values, blocks in a random order."""
    B, Hkv, d, bs, fmt = case["B"], case["Hkv"], case["d"], case["block"], case["fmt"]
    blocks = [-(-t // bs) for t in n_tokens]
    width = max(1, max(blocks) + 1)
    n_blocks = sum(blocks) + spare
    order = torch.randperm(n_blocks, generator=g, device=DEV).to(torch.int32)
    code = torch.int8 if fmt == "int8" else torch.float8_e4m3fn
    k = torch.zeros((n_blocks, Hkv, bs, d), dtype=torch.uint8, device=DEV).view(code)
    v = torch.zeros((n_blocks, Hkv, bs, d), dtype=torch.uint8, device=DEV).view(code)
    ks = torch.ones((n_blocks, Hkv), device=DEV)
    vs = torch.ones((n_blocks, Hkv), device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    mu = torch.randn((256, d), generator=g, device=DEV)
    at = 0
    for b in range(B):
        nb = blocks[b]
        if nb == 0:
            continue
        ids = order[at: at + nb].long()
        at += nb
        table[b, :nb] = ids.to(torch.int32)
        for j in range(0, nb, 512):
            sub = ids[j: j + 512]
            shape = (sub.numel(), Hkv, bs)
            lab = torch.randint(0, 256, shape, generator=g, device=DEV)
            x = mu[lab] + 0.3 * torch.randn((*shape, d), generator=g, device=DEV)
            c, s = _quantise(x, fmt)
            k.view(torch.uint8)[sub], ks[sub] = c.view(torch.uint8), s
            c, s = _quantise(torch.randn((*shape, d), generator=g, device=DEV), fmt)
            v.view(torch.uint8)[sub], vs[sub] = c.view(torch.uint8), s
    length = torch.tensor(list(n_tokens), dtype=torch.int32, device=DEV)
    return dict(k=k, v=v, ks=ks, vs=vs, table=table, len=length, order=order, used=at, mu=mu, block=bs, fmt=fmt)


def _queries(case, mu, g):
    q = torch.randn((case["B"], case["Hq"], case["d"]), generator=g, device=DEV)
    pick = torch.randint(0, mu.shape[0], (case["B"], case["Hq"]), generator=g, device=DEV)
    return (0.5 * mu[pick] + q).to(_dtype(case))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    n, add = _lengths(case)
    if op == "plan":
        st = _plan_state(case, n, add, g)
    elif op == "append":
        st = _append_state(case, n, add, g)
    else:
        st = _pool(case, n, g, 0)
        st["q"] = _queries(case, st["mu"], g)
        st["Hkv"] = case["Hkv"]
        if op == "sparse":
            G = case["Hkv"] if case["mode"] == "group" else case["Hq"]
            U, T = case["B"] * G, case["T"]
            rank = torch.rand((U, T), generator=g, device=DEV)
            rank[:, : min(4, T)] = -1.0  # the sinks come first
            st["tok"] = rank.argsort(dim=1)[:, : case["n"]].to(torch.int32).contiguous()
            st["n_tok"] = torch.tensor(_entries(case), dtype=torch.int32, device=DEV)
            st["G"] = G
    st["op"] = op
    if own:
        _handles(case, st)
    return st


def _plan_state(case, n, add, g):
    """Requests that already hold their new tokens: a pass gives those back and takes slots for them again."""
    bs, B = case["block"], case["B"]
    full = [x + a for x, a in zip(n, add)]
    blocks = [-(-x // bs) for x in full]
    n_blocks = sum(blocks) + 3
    order = torch.randperm(n_blocks, generator=g, device=DEV).to(torch.int32)
    width = max(blocks) + 2
    J = torch.arange(width, device=DEV)[None, :]
    nb = torch.tensor(blocks, device=DEV)
    first = torch.cumsum(nb, 0) - nb
    at = (first[:, None] + J).clamp_max(n_blocks - 1)
    table = torch.where(J < nb[:, None], order[at], torch.full_like(order[at], -1)).contiguous()
    free = torch.cat([order[sum(blocks):], torch.full((sum(blocks),), -1, dtype=torch.int32, device=DEV)])
    return dict(block=bs, table=table, len=torch.tensor(full, dtype=torch.int32, device=DEV), free=free,
                n_free=torch.full((1,), 3, dtype=torch.int32, device=DEV),
                up=torch.tensor(add, dtype=torch.int32, device=DEV),
                down=torch.tensor([-a for a in add], dtype=torch.int32, device=DEV), rows=sum(add))


def _append_state(case, n, add, g):
    bs, B, Hkv, d = case["block"], case["B"], case["Hkv"], case["d"]
    full = [x + a for x, a in zip(n, add)]
    st = _pool(case, full, g, 2)
    N = sum(add)
    st["start"] = torch.tensor([sum(add[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
    st["granted"] = torch.tensor(add, dtype=torch.int32, device=DEV)
    b = torch.repeat_interleave(torch.arange(B, device=DEV), st["granted"].long())
    pos = torch.arange(N, device=DEV) - st["start"].long()[b] + torch.tensor(n, device=DEV)[b]
    st["slot"] = (st["table"][b, pos // bs].long() * bs + pos % bs).to(torch.int32)
    lab = torch.randint(0, 256, (N, Hkv), generator=g, device=DEV)
    st["k_new"] = (st["mu"][lab] + 0.3 * torch.randn((N, Hkv, d), generator=g, device=DEV)).to(_dtype(case))
    st["v_new"] = torch.randn((N, Hkv, d), generator=g, device=DEV).to(_dtype(case))
    # read back: each request from the start of the first block that the new rows touch
    st["first"] = torch.tensor([x // bs * bs for x in n], dtype=torch.int32, device=DEV)
    st["R"] = max(f - x // bs * bs for f, x in zip(full, n))
    st["k_out"] = torch.empty((B, Hkv, st["R"], d), dtype=_dtype(case), device=DEV)
    st["v_out"] = torch.empty_like(st["k_out"])
    return st


def _handles(case, st):
    """The framework's descriptors and workspaces over the state's tensors."""
    import graph_community_sparse_b200 as ckv
    if st["op"] == "plan":
        st["cache"] = ckv.block_table(st["table"], st["len"], st["free"], st["n_free"], st["block"])
        st["p_down"], st["p_up"] = ckv.new_plan(st["cache"], 0), ckv.new_plan(st["cache"], st["rows"])
        return
    st["cache"] = ckv.q8_cache(st["k"], st["v"], st["ks"], st["vs"], st["table"], st["len"], case.get("Hq", case["Hkv"]),
                               _dtype(case))
    if st["op"] == "append":
        st["plan"] = ckv.Plan(st["start"], st["slot"], st["granted"])
        return
    st["out"] = torch.empty(st["q"].shape, device=DEV)
    if st["op"] == "dense":
        st["ws"] = ckv.new_workspace(ckv.ckv_q8_workspace_size(st["cache"]))
        return
    shape = ckv.q8_shape(st["cache"], case["T"])
    st["graph"] = ckv.new_graph(shape, ckv.PER_GROUP if case["mode"] == "group" else ckv.PER_HEAD, min(4, case["T"]), 1, 0)
    st["sel"] = ckv.new_selection(shape, st["graph"], case["n"])
    st["sel"].sel_tok.copy_(st["tok"])
    st["sel"].n_tok.copy_(st["n_tok"])
    st["ws"] = ckv.new_workspace(ckv.ckv_q8_workspace_size(st["cache"], st["graph"], st["sel"]))


# ---------------------------------------------------------------------------
# a pass
# ---------------------------------------------------------------------------

def run(st):
    op = st["op"]
    if own:
        import graph_community_sparse_b200 as ckv
        if op == "plan":
            ckv.ckv_plan_blocks(st["cache"], st["down"], st["p_down"])
            ckv.ckv_plan_blocks(st["cache"], st["up"], st["p_up"])
            p = st["p_up"]
            return dict(table=st["table"], len=st["len"], free=st["free"], n_free=st["n_free"], start=p.start, slot=p.slot,
                        granted=p.granted)
        if op == "append":
            ckv.ckv_quant_append(st["cache"], st["plan"], st["k_new"], st["v_new"])
            ckv.ckv_q8_read(st["cache"], st["k_out"], st["v_out"], st["first"])
            return dict(k=st["k_out"], v=st["v_out"], ks=st["ks"], vs=st["vs"])
        if op == "dense":
            ckv.ckv_dense_decode_q8(st["cache"], st["q"], st["out"], st["ws"])
        else:
            ckv.ckv_sparse_decode_q8(st["cache"], st["q"], st["graph"], st["sel"], st["out"], None, st["ws"])
        return st["out"]
    if op == "plan":
        _plain_plan(st, st["down"], 0)
        start, slot, granted = _plain_plan(st, st["up"], st["rows"])
        return dict(table=st["table"], len=st["len"], free=st["free"], n_free=st["n_free"], start=start, slot=slot,
                    granted=granted)
    if op == "append":
        _plain_append(st)
        k, v = _plain_read(st)
        return dict(k=k, v=v, ks=st["ks"], vs=st["vs"])
    return _plain_dense(st) if op == "dense" else _plain_sparse(st)


def _blocks(n, bs):
    return (n + bs - 1) // bs


def _plain_plan(st, add, rows):
    """Shrinks, then grows; integers throughout.  Updates table, len, free and n_free in place."""
    bs, table, length, free, n_free = st["block"], st["table"], st["len"], st["free"], st["n_free"]
    B, width = table.shape
    J = torch.arange(width, device=DEV)[None, :]
    n0 = length.long()
    n1 = n0 - torch.minimum((-add.long()).clamp_min(0), n0)
    # blocks without a token go onto the free list, the last one in request order lowest
    gone = (J >= _blocks(n1, bs)[:, None]) & (J < _blocks(n0, bs)[:, None])
    k = torch.cumsum(gone.reshape(-1), 0).reshape(gone.shape) - 1
    freed = gone.sum()
    room = torch.cat([free, free[:1]])
    room.scatter_(0, torch.where(gone, n_free.long() + freed - 1 - k, torch.full_like(k, free.numel())).reshape(-1), table.reshape(-1))
    avail = n_free.long() + freed
    # growth: within the table's width and the slot map, and while the free blocks last
    up = add.long().clamp_min(0)
    start = torch.cat([torch.zeros_like(up[:1]), torch.cumsum(up, 0)])
    fits = (n1 + up <= width * bs) & (start[1:] <= rows)
    need = torch.where(fits, _blocks(n1 + up, bs) - _blocks(n1, bs), torch.zeros_like(up))
    ok = fits & ((need == 0) | (torch.cumsum(need, 0) <= avail))
    grown = torch.where(ok, up, torch.zeros_like(up))
    n2 = n1 + grown
    new = (J >= _blocks(n1, bs)[:, None]) & (J < _blocks(n2, bs)[:, None])
    k = torch.cumsum(new.reshape(-1), 0).reshape(new.shape) - 1
    took = room[(avail - 1 - k).clamp(0, free.numel() - 1)]
    table.copy_(torch.where(new, took, torch.where(gone, torch.full_like(table, -1), table)))
    length.copy_(n2)
    free.copy_(room[:-1])
    n_free.copy_(avail - new.sum())
    row = torch.arange(rows, device=DEV)
    b = torch.searchsorted(start[1:].contiguous(), row, right=True).clamp_max(B - 1)
    pos = n1[b] + row - start[b]
    held = ok[b] & (row < start[-1])
    at = table[b, torch.where(held, pos // bs, torch.zeros_like(pos))].long()
    slot = torch.where(held, at * bs + pos % bs, torch.full_like(pos, -1))
    return start.to(torch.int32), slot.to(torch.int32), (n2 - n0).to(torch.int32)


def _plain_append(st):
    bs, fmt = st["block"], st["fmt"]
    slot, start = st["slot"].long(), st["start"].long()
    blk = slot // bs
    lead = blk[start[:-1]]      # each request's first touched block: the one that may hold older rows
    before = slot[start[:-1]] % bs
    for codes, scales, new in ((st["k"], st["ks"], st["k_new"]), (st["v"], st["vs"], st["v_new"])):
        x = new.float()
        amax = torch.zeros_like(scales).scatter_reduce_(0, blk[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        fresh = _scale(amax.clamp_min(FLOOR), fmt)
        old = scales[lead]
        keep = torch.where((before > 0)[:, None], torch.maximum(old, fresh[lead]), fresh[lead])
        fresh[lead] = keep
        # older rows of the first block, on the new scale
        ratio = old * (1.0 / keep)
        rows = _times(codes[lead].float(), ratio[..., None, None], fmt)
        is_old = (torch.arange(bs, device=DEV)[None, :] < before[:, None])[:, None, :, None]
        codes.view(torch.uint8)[lead] = torch.where(is_old, rows.view(torch.uint8), codes[lead].view(torch.uint8))
        inv = 1.0 / fresh[blk]
        codes.view(torch.uint8)[blk, :, slot % bs] = _times(x, inv[..., None], fmt).view(torch.uint8)
        scales[blk] = fresh[blk]


def _times(x, f, fmt):
    """Codes of x f, the product exact: it lies next to a rounding border often (x = amax/2)."""
    if fmt == "int8":
        return (x.double() * f.double()).round().clamp(-127, 127).to(torch.int8)
    return (x * f).to(torch.float8_e4m3fn)  # f is a power of two


def _plain_read(st):
    bs, R = st["block"], st["R"]
    pos = st["first"].long()[:, None] + torch.arange(R, device=DEV)[None, :]
    inside = pos < st["len"].long()[:, None]
    blk = st["table"].gather(1, torch.where(inside, pos, torch.zeros_like(pos)) // bs).long().clamp_min(0)
    out = []
    for codes, scales in ((st["k"], st["ks"]), (st["v"], st["vs"])):
        x = codes.view(torch.uint8)[blk, :, pos % bs].view(codes.dtype).float() * scales[blk][..., None]
        x = torch.where(inside[:, :, None, None], x, torch.zeros_like(x))
        out.append(x.permute(0, 2, 1, 3).to(st["k_out"].dtype).contiguous())
    return out


def _values(codes, scales, ids):
    return codes.view(torch.uint8)[ids].view(codes.dtype).float() * scales[ids][..., None, None]


def _softmax(x):
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_dense(st):
    bs = st["block"]
    B, Hq, d = st["q"].shape
    Hkv = st["Hkv"]
    ids = st["table"].long().clamp_min(0)  # [B, width]
    T = ids.shape[1] * bs
    k = _values(st["k"], st["ks"], ids).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T, d)
    x = torch.matmul(st["q"].float().reshape(B, Hkv, Hq // Hkv, d), k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    del k
    held = torch.arange(T, device=DEV)[None, :] < st["len"].long()[:, None]
    p = _softmax(x.masked_fill(~held[:, None, None, :], float("-inf")))
    v = _values(st["v"], st["vs"], ids).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T, d)
    return torch.matmul(p, v).reshape(B, Hq, d)


def _plain_sparse(st):
    bs, G, Hkv = st["block"], st["G"], st["Hkv"]
    B, Hq, d = st["q"].shape
    U = B * G
    u = torch.arange(U, device=DEV)
    head = (u % G) // (G // Hkv)
    pos = st["tok"].long()
    blk = st["table"].long()[(u // G)[:, None], pos // bs]
    at = (blk, head[:, None].expand_as(blk), pos % bs)
    k = st["k"].view(torch.uint8)[at].view(st["k"].dtype).float() * st["ks"][at[:2]][..., None]
    v = st["v"].view(torch.uint8)[at].view(st["v"].dtype).float() * st["vs"][at[:2]][..., None]
    x = torch.matmul(st["q"].float().reshape(U, Hq // G, d), k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    held = torch.arange(pos.shape[1], device=DEV)[None, :] < st["n_tok"].long()[:, None]
    return torch.matmul(_softmax(x.masked_fill(~held[:, None, :], float("-inf"))), v).reshape(B, Hq, d)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers only
    st = prepare(case, seed)
    bs, table, length = case["block"], st["table"].long(), st["len"].tolist()
    if case["op"] == "append":
        return _exact_append(case, st)
    B, Hq, d = st["q"].shape
    Hkv = case["Hkv"]
    out = torch.zeros((B, Hq, d), dtype=torch.float64, device=DEV)
    q = st["q"].double()
    r = Hq // Hkv
    for b in range(B):
        for h in range(Hkv):
            t = torch.arange(length[b], device=DEV)
            blk, row = table[b, t // bs], t % bs
            k = st["k"][:, h].view(torch.uint8)[blk, row].view(st["k"].dtype).double() * st["ks"][blk, h].double()[:, None]
            v = st["v"][:, h].view(torch.uint8)[blk, row].view(st["v"].dtype).double() * st["vs"][blk, h].double()[:, None]
            x = (q[b, h * r: (h + 1) * r] @ k.T) / math.sqrt(d)  # [r, tokens]
            if case["op"] == "sparse":
                keep = torch.zeros_like(x, dtype=torch.bool)
                for i in range(r):
                    unit = b * st["G"] + (h if case["mode"] == "group" else h * r + i)
                    keep[i, st["tok"][unit, : int(st["n_tok"][unit])].long()] = True
                x = x.masked_fill(~keep, float("-inf"))
            out[b, h * r: (h + 1) * r] = torch.softmax(x, dim=-1) @ v
    return out


def _exact_append(case, st):
    """Block by block: the largest new magnitude sets the scale (never below what the block's older rows have), each
    value goes to the nearest code, ties to the even one."""
    bs, fmt, B = case["block"], case["fmt"], case["B"]
    n, add = _lengths(case)
    start = 0
    R = st["R"]
    outs = {}
    for name, codes, scales, new in (("k", st["k"], st["ks"], st["k_new"]), ("v", st["v"], st["vs"], st["v_new"])):
        s_out = scales.double().clone()
        values = torch.zeros((B, case["Hkv"], R, case["d"]), dtype=torch.float64, device=DEV)
        start = 0
        for b in range(B):
            first = n[b] // bs * bs
            total = n[b] + add[b] - first
            nb = -(-total // bs)
            ids = st["table"][b, first // bs: first // bs + nb].long()
            old = n[b] - first
            x = torch.zeros((nb * bs, case["Hkv"], case["d"]), dtype=torch.float64, device=DEV)
            x[old: total] = new[start: start + add[b]].double()
            start += add[b]
            x = x.reshape(nb, bs, case["Hkv"], case["d"]).permute(0, 2, 1, 3)  # [nb, Hkv, bs, d]
            amax = x.abs().amax(dim=(2, 3)).clamp_min(FLOOR)
            if fmt == "int8":
                s = (amax / 127).float().double()
            else:
                s = torch.exp2(torch.ceil(torch.log2(amax / 448)))
            if old:
                s[0] = torch.maximum(s[0], scales[ids[0]].double())
            inv = (1 / s).float().double()
            y = x * inv[..., None, None]
            if old:
                ratio = (scales[ids[0]].double() * inv[0]).float().double()
                c = codes[ids[0]].view(torch.uint8)[:, :old].contiguous().view(codes.dtype).double()
                y[0, :, :old] = c * ratio[:, None, None]
            y = y.round().clamp(-127, 127) if fmt == "int8" else y.float().to(torch.float8_e4m3fn).double()
            s_out[ids] = s
            y = (y * s[..., None, None]).permute(1, 0, 2, 3).reshape(case["Hkv"], nb * bs, case["d"])
            values[b, :, :total] = y[:, :total]
        outs[name], outs[name + "s"] = values, s_out
    return dict(k=outs["k"], v=outs["v"], ks=outs["ks"], vs=outs["vs"])
