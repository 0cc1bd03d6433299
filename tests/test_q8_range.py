"""The 8-bit attention's arithmetic over the range of its formats: what the bounds of the other tests are too wide to
see.  Scores where one channel of the keys is large, scales that differ by more than fp32's exponents, values that are not
finite behind small weights, and the size of the rounding errors themselves."""
import ctypes
import math
import random

import numpy as np
import pytest
import torch

import graph_community_sparse_b200 as ckv
import q8_ref as Q
from parity_util import check_neighbours
from test_abi import FAKE, UNSUPPORTED
from test_q8_abi import _q8, _table

DEV = "cuda"


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def pool(lens, Hkv, gq, d, block, fmt, dtype, seed=0):
    """Requests of these lengths in a pool of zeros, blocks in random order; scales of 1/100."""
    nb = [-(-n // block) for n in lens]
    cache = ckv.new_q8_cache(len(lens), Hkv, Hkv * gq, d, sum(nb) + 2, block, max(nb + [1]), fmt, dtype)
    ids = list(range(sum(nb) + 2))
    random.Random(seed).shuffle(ids)
    for b, n in enumerate(nb):
        cache.table[b, :n] = i32([ids.pop() for _ in range(n)])
    cache.len.copy_(i32(lens))
    cache.k_scale.fill_(0.01)
    cache.v_scale.fill_(0.01)
    return cache


def put(cache, which, b, values):
    """Codes [n, Hkv, d] of request b."""
    t, n, bs = getattr(cache, which), values.shape[0], cache.desc.blocks.block
    ids = cache.table[b].tolist()
    for j in range(0, n, bs):
        t[ids[j // bs], :, : min(bs, n - j)] = values[j: j + bs].transpose(0, 1).to(DEV).to(t.dtype)


def held(cache, b, h):
    """K and V values of request b, head h, in float64 [n, d]."""
    n, bs = int(cache.len[b]), cache.desc.blocks.block
    ids = cache.table[b, : -(-n // bs)].long()
    out = []
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = t[ids, h].float().double() * s[ids, h].double()[:, None, None]
        out.append(x.reshape(-1, t.shape[-1])[:n].cpu().numpy())
    return out


def every_way(cache, q, S=0, neighbours=False, shuffle=True):
    """The outputs of the dense call and of lists of all tokens, in random order or in theirs (one a query head, one a KV
    head), and the last one's lists and neighbours."""
    B = cache.B
    outs, lists, nbr = [], None, None
    out = torch.full(q.shape, float("nan"), device=DEV)
    ckv.ckv_dense_decode_q8(cache, q, out, ckv.new_workspace(ckv.ckv_q8_workspace_size(cache)))
    outs.append(out)
    lens = cache.len.tolist()
    for mode in (ckv.PER_HEAD, ckv.PER_GROUP):
        shape = ckv.q8_shape(cache, max(lens))
        graph = ckv.new_graph(shape, mode, S, 1, 0)
        sel = ckv.new_selection(shape, graph, max(lens))
        G = graph.U // B
        lists = [random.Random(u).sample(range(lens[u // G]), lens[u // G]) if shuffle else list(range(lens[u // G]))
                 for u in range(graph.U)]
        for u, x in enumerate(lists):
            sel.sel_tok[u, : len(x)] = i32(x)
        sel.n_tok.copy_(i32([len(x) for x in lists]))
        out = torch.full(q.shape, float("nan"), device=DEV)
        nbr = torch.empty((graph.U, 8), dtype=torch.int32, device=DEV) if neighbours else None
        ckv.ckv_sparse_decode_q8(cache, q, graph, sel, out, nbr,
                                 ckv.new_workspace(ckv.ckv_q8_workspace_size(cache, graph, sel)))
        outs.append(out)
    return outs, lists, nbr


def score_share(S):
    """The part of a weight's relative error that its score brings: q and the codes are exact in fp16 (bf16 q), at most
    d/16 = 8 products of 16 terms are added with an error of 2^-23 of the largest sum each (two chains of four, a
    truncating accumulator), then the chains' sum, the scale's two products and the subtraction: 14 * 2^-23 S, with S the
    largest sum of |q_i k_i| / sqrt(d)."""
    return 14 * 2.0 ** -23 * S


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d,gq", [(128, 4), (128, 8), (64, 1), (64, 2), (64, 8)])
@pytest.mark.parametrize("nonzeros", [1, 4, 60])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weights_beside_a_large_channel(fmt, d, gq, nonzeros, dtype):
    """One channel of the keys takes the codes' whole range and q is zero there; a few others are 1 or -1 and the rest 0.
    V is the identity, so that the output is the weights themselves: their errors follow the scores' sums of |q k|, not
    the codes' range."""
    n, gen = d, torch.Generator().manual_seed(d + gq + nonzeros)
    cache = pool([n], 1, gq, d, 16, fmt, dtype)
    put(cache, "v", 0, 100 * torch.eye(n)[:, None, :])
    cache.k_scale.fill_(16.0)
    for again in range(8):
        k = torch.zeros((n, 1, d))
        at = torch.rand((n, 1, d), generator=gen).topk(nonzeros, -1).indices
        k.scatter_(2, at, 1.0 - 2 * torch.randint(0, 2, (n, 1, nonzeros), generator=gen).float())
        k[:, 0, 5] = 120.0
        put(cache, "k", 0, k)
        q = torch.randn((1, gq, d), generator=gen).bfloat16().to(dtype)  # exact in one fp16 term, whatever the type
        q[:, :, 5] = 0.0
        q = q.to(DEV)
        outs, lists, nbr = every_way(cache, q, neighbours=True)
        K, V = held(cache, 0, 0)
        for h in range(gq):
            want, S = Q.attention(q[0, h].double().cpu().numpy(), K, V)
            # beside the scores: exp2 2^-22, a weight in two fp16 terms 2^-22 (from 2^-6 of the largest on), scale
            # products 2^-23, and the weights' sum over 5 tiles, 8 lanes and 4 warps; numerator and denominator
            rel = 2 * (score_share(S) + 2 * 2.0 ** -22 + 2.0 ** -23 * (1 + 5 + 8 + 4))
            large = want >= want.max() / 64
            for out in outs:
                err = np.abs(out[0, h].double().cpu().numpy() / want - 1)[large].max()
                assert err <= rel, (again, h, err, rel)
        qn = q[0].double().cpu().numpy()
        S = (np.abs(K) @ np.abs(qn).T).max() / math.sqrt(d)
        check_neighbours(nbr[0].tolist(), qn, K, np.asarray(lists[0]), 0, band=2 * score_share(S))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d,gq", [(64, 4), (128, 8), (64, 1)])
@pytest.mark.parametrize("score", [0.0, -80.0, -300.0])
@pytest.mark.parametrize("which", ["k", "v"])
def test_not_finite_blocks_reach_the_output_behind_any_weight(fmt, d, gq, score, which):
    """A block whose scale is NaN, for K or V of one head, makes its request's outputs of that head NaN, even where its
    tokens weigh 2^-115 or nothing in fp32; no other output."""
    n = 100
    cache = pool([n, n], 2, gq, d, 16, fmt, torch.float32)
    k = torch.zeros((n, 2, d))
    k[48:64, :, 3] = -96.0
    for b in range(2):
        put(cache, "k", b, k)
        put(cache, "v", b, torch.full((n, 2, d), 5.0))
    at = int(cache.table[0, 3])
    cache.k_scale[at] = -score * math.sqrt(d) / 96
    (cache.k_scale if which == "k" else cache.v_scale)[at, 1] = float("nan")
    q = torch.zeros((2, 2 * gq, d), device=DEV)
    q[:, :, 3] = 1.0
    for out in every_way(cache, q)[0]:
        assert torch.isnan(out[0, gq:]).all()
        assert torch.isfinite(out[0, :gq]).all() and torch.isfinite(out[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d,gq", [(64, 4), (128, 8), (128, 1)])
@pytest.mark.parametrize("v_scales", [(2.0 ** 14, 0.0), (2.0 ** 60, 2.0 ** -107 / 127), (2.0 ** 90, 1.0), (0.0, 2.0 ** 14),
                                      (2.0 ** -100, 2.0 ** 100)])
def test_v_scales_that_fall_or_rise_where_the_scores_jump(fmt, d, gq, v_scales):
    """A request whose second half scores 150 to 300 (in powers of two) above its first, and whose V scale there is that
    much smaller, zero or larger: finite, and the second half's values."""
    n = 192  # one block's warps see tiles of the first half, then of the second
    cache = pool([n], 1, gq, d, 32, fmt, torch.float32)
    k = torch.zeros((n, 1, d))
    k[96:, :, 0] = 64.0
    put(cache, "k", 0, k)
    gen = torch.Generator().manual_seed(1)
    put(cache, "v", 0, torch.randint(-60, 61, (n, 1, d), generator=gen).float().div(8).round().mul(8))
    for j in range(6):
        cache.v_scale[int(cache.table[0, j])] = v_scales[j // 3]
    for step in (150.0, 300.0):
        cache.k_scale.fill_(step * math.log(2) * math.sqrt(d) / 64)
        q = torch.zeros((1, gq, d), device=DEV)
        q[:, :, 0] = 1.0
        K, V = held(cache, 0, 0)
        want = V[96:].mean(0)  # equal weights; the first half's are 2^-150 of them or less
        rest = 2.0 ** -step * np.abs(V[:96]).max()
        # 96 equal weights: each and their sums off by at most 2^-21 (exp2, two fp16 terms, scale products, sums over
        # 3 tiles and 4 warps), twice for numerator and denominator
        tol = 2 * 2.0 ** -21 * np.abs(V[96:]).max() + 2 * rest
        for out in every_way(cache, q, shuffle=False)[0]:
            assert torch.isfinite(out).all()
            assert np.abs(out.double().cpu().numpy() - want).max() <= tol


# ---------------------------------------------------------------------------
# the size of the rounding errors
# ---------------------------------------------------------------------------

def rms_tol(S):
    """Bound of the outputs' error relative to their size, both as root mean squares, for V of mean zero that knows
    nothing of the errors: an error of at most e in each weight moves an output by e sqrt(sum w^2) sigma, which is e
    times the output's own size.  e: the score's share, exp2 and the two fp16 terms of a weight 2^-22 each, and 2^-20 for
    the scale products and the sums in fp32 (a few dozen additions, each 2^-24 of a partial sum).  The weights' sum has
    at most the same error, apart from it: sqrt(2)."""
    return math.sqrt(2) * (score_share(S) + 2 * 2.0 ** -22 + 2.0 ** -20)


def relative_rms(got, want):
    return float(((got - want) ** 2).mean() ** 0.5 / (want ** 2).mean() ** 0.5)


def in_two(x, terms):
    """x as a sum of fp16 terms."""
    hi = x.astype(np.float16).astype(np.float64)
    return hi if terms == 1 else hi + (x - hi).astype(np.float16).astype(np.float64)


@pytest.mark.parametrize("n", [33, 1000])
@pytest.mark.parametrize("q_terms,w_terms", [(2, 2), (1, 2), (2, 1)])
def test_the_bound_sees_a_lost_term(n, q_terms, w_terms):
    """The kernel's fp16 splits of q and of the weights modelled in float64: the bound holds with both terms and fails
    where either lo term is dropped, which the wider bounds of the other tests would let pass."""
    rng = np.random.default_rng(n)
    d, H = 128, 64
    k, v = rng.integers(-127, 128, (2, n, d)) / 73.0
    q = (0.1 * rng.standard_normal((H, d))).astype(np.float32).astype(np.float64)
    top = np.exp2(np.floor(np.log2(np.abs(q).max(1, keepdims=True))) - 14)
    got, want, S = [], [], 0.0
    for h in range(H):
        o, s = Q.attention(q[h], k, v)
        w = np.exp(k @ (in_two(q[h] / top[h], q_terms) * top[h]) / math.sqrt(d))
        w = in_two(w * 32 / w.max(), w_terms)
        got.append(w @ v / w.sum())
        want.append(o)
        S = max(S, s)
    err = relative_rms(np.array(got), np.array(want))
    assert (err <= rms_tol(S)) == (q_terms == w_terms == 2), (err, rms_tol(S))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,gq", [(64, 8), (128, 4), (128, 8), (64, 2)])
@pytest.mark.parametrize("n", [33, 200, 1000, 5000, 70000])
def test_rounding_errors_keep_their_size(fmt, dtype, d, gq, n):
    Hkv = 2
    cache = pool([n], Hkv, gq, d, 64, fmt, dtype)
    gen = torch.Generator(device=DEV).manual_seed(n + d + gq)
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = torch.randint(-127, 128, t.shape, generator=gen, device=DEV, dtype=torch.int32).to(torch.float32)
        t.copy_(x.to(t.dtype))
        s.copy_((1 + torch.rand(s.shape, generator=gen, device=DEV)) / 100)
    q = (0.1 * torch.randn((1, Hkv * gq, d), generator=gen, device=DEV)).to(dtype)
    outs, _, _ = every_way(cache, q)
    ids = cache.table[0].long()
    K, V = ((t[ids].float().double() * s[ids].double()[:, :, None, None]).transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
            for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    qd = q[0].double().view(Hkv, gq, d)
    want = torch.softmax(torch.einsum("hgd,htd->hgt", qd, K) / math.sqrt(d), -1) @ V
    S = float((torch.einsum("hgd,htd->hgt", qd.abs(), K.abs()) / math.sqrt(d)).max())
    for out in outs:
        err = relative_rms(out[0].double().view(Hkv, gq, d), want)
        assert err <= rms_tol(S), (err, rms_tol(S))


# ---------------------------------------------------------------------------
# long lists
# ---------------------------------------------------------------------------

def check_permuted(cache, q, S_sinks, neighbours):
    """Lists of all of a request's tokens in random order, a list a KV head, against the dense reference in float64; the
    neighbours' logits against the eight largest."""
    lens = cache.len.tolist()
    B, Hkv, Hq, d = cache.B, cache.Hkv, cache.Hq, cache.d
    cap, gq = max(lens), Hq // Hkv
    shape = ckv.q8_shape(cache, cap)
    graph = ckv.new_graph(shape, ckv.PER_GROUP, S_sinks, 1, 0)
    sel = ckv.new_selection(shape, graph, cap)
    gen = torch.Generator(device=DEV).manual_seed(1)
    for u in range(graph.U):
        n = lens[u // Hkv]
        sel.sel_tok[u, :n] = torch.randperm(n, generator=gen, device=DEV).to(torch.int32)
    sel.n_tok.copy_(i32([lens[u // Hkv] for u in range(graph.U)]))
    out = torch.full(q.shape, float("nan"), device=DEV)
    nbr = torch.full((graph.U, 8), -7, dtype=torch.int32, device=DEV) if neighbours else None
    ws = ckv.new_workspace(ckv.ckv_q8_workspace_size(cache, graph, sel))
    for _ in range(2):
        ckv.ckv_sparse_decode_q8(cache, q, graph, sel, out, nbr, ws)
    assert not ws[256: 256 + 8192 * 4].any()  # the counters are zero again
    for b, n in enumerate(lens):
        if n == 0:
            assert not out[b].any()
            continue
        ids = cache.table[b, : -(-n // cache.desc.blocks.block)].long()
        K, V = ((t[ids].float().double() * s[ids].double()[:, :, None, None]).transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
                for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        qd = q[b].double().view(Hkv, gq, d)
        x = torch.einsum("hgd,htd->hgt", qd, K) / math.sqrt(d)
        S = float((torch.einsum("hgd,htd->hgt", qd.abs(), K.abs()) / math.sqrt(d)).max())
        tol = Q.attention_tol(S, n, float(V.abs().max()))
        assert float((out[b].double().view(Hkv, gq, d) - torch.softmax(x, -1) @ V).abs().max()) <= tol
        for h in range(Hkv if neighbours else 0):
            u, best = b * Hkv + h, x[h].amax(0)
            skipped = sel.sel_tok[u, : min(S_sinks, n)].long()  # the list's first entries take the sinks' places
            best[skipped] = -math.inf
            m = min(8, n - len(skipped))
            got = nbr[u].tolist()
            assert len(set(got[:m])) == m and got[m:] == [-1] * (8 - m)
            if m:
                cut = float(best.topk(m).values[-1])
                assert float(best[torch.tensor(got[:m], device=DEV)].min()) >= cut - 2 * score_share(S)


def random_pool(lens, Hkv, gq, d, block, fmt, dtype, seed):
    cache = pool(lens, Hkv, gq, d, block, fmt, dtype, seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = torch.randint(-127, 128, t.shape, generator=gen, device=DEV, dtype=torch.int32).to(torch.float32)
        t.copy_(x.to(t.dtype))
        s.copy_((1 + torch.rand(s.shape, generator=gen, device=DEV)) / 100)
    return cache, torch.randn((len(lens), Hkv * gq, d), generator=gen, device=DEV).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("lens", [[1023, 1024, 1025, 192, 193], [4095, 4097, 4096], [32767, 16], [32768], [32769, 50000]])
def test_lists_where_the_least_piece_changes(lens, neighbours):
    """Lists of 12, 64, 256 and 2048 tiles and their neighbours."""
    cache, q = random_pool(lens, 1, 4, 64, 64, "int8", torch.float32, len(lens))
    check_permuted(cache, q, 0, neighbours)


@pytest.mark.gpu
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("gq,d,fmt", [(1, 64, "int8"), (8, 64, "e4m3"), (4, 128, "int8")])
def test_lists_laid_end_to_end(gq, d, fmt, neighbours):
    """More lists than blocks of the grid, a few so long that many blocks share them, some empty."""
    lens = [100 + b % 37 for b in range(330)]
    lens[3], lens[100], lens[101], lens[329] = 30000, 9000, 20001, 25000
    for b in range(5, 330, 11):
        lens[b] = 0
    cache, q = random_pool(lens, 2, gq, d, 32, fmt, torch.bfloat16, gq)
    check_permuted(cache, q, 2, neighbours)


# ---------------------------------------------------------------------------
# sizes of the read, without a GPU
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hkv", [(512, 8), (8192, 1), (1023, 8)])
def test_read_sizes_past_the_grid_are_refused(d, B, Hkv):
    """Past the documented bound, B Hkv ceil(R d / 2048) < 2^31, the host refuses (nothing is launched)."""
    cache = _q8(_table(B=B, n_blocks=100), Hkv=Hkv, Hq=4 * Hkv, d=d)
    for R in (-(-2 ** 31 // (B * Hkv)) * (2048 // d), 2 ** 30):
        assert ckv.lib.ckv_q8_read(ctypes.byref(cache), None, R, FAKE, FAKE, 0, 0, d, None) == UNSUPPORTED
        assert "2^31" in ckv.ckv_last_error()
