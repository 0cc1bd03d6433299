"""Community graphs over the paged 8-bit cache when its requests do not all start alike and simply grow: growth refused
after a token has joined, idle requests, tokens given back, requests that end, requests of different length and new ones.
A join that is undone leaves no trace, which is compared bit for bit with the state before it; no position is ever
attended twice."""
import ctypes
import re

import numpy as np
import pytest
import torch

import graph_community_sparse_b200 as ckv
import q8_ref as Q
from graph_community_sparse_b200.layer import PagedLayerState
from test_abi import CAPACITY, FAKE, HEADER, INVALID, WORKSPACE, _graph, _sel
from test_q8_abi import _q8, _table

DEV = "cuda"
R = ctypes.byref
FIELDS = ("comm_of", "offs", "cnt", "cent", "cent_q", "cent_qs", "num_comm", "tail_len", "built")


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------
# without a GPU
# ---------------------------------------------------------------------------

TRIMS = [
    ("cache", lambda: (_q8(d=96), _graph()), "unsupported"),
    ("graph mode", lambda: (_q8(), _graph(mode=2, undo=FAKE, built=FAKE)), INVALID),
    ("graph T_cap", lambda: (_q8(), _graph(T_cap=8192, undo=FAKE, built=FAKE)), CAPACITY),
    ("no undo", lambda: (_q8(), _graph(built=FAKE)), INVALID),
    ("no built", lambda: (_q8(), _graph(undo=FAKE)), INVALID),
]


@pytest.mark.parametrize("name,make,status", TRIMS, ids=[t[0] for t in TRIMS])
def test_trim_refusals(name, make, status):
    cache, graph = make()
    got = ckv.lib.ckv_trim_graph_q8(R(cache), R(graph), None)
    assert got == (3 if status == "unsupported" else status), ckv.ckv_last_error()
    assert ckv.ckv_last_error()


def _build(cache=None, graph=None, labels=FAKE, stride=4096, T=4096, ws=FAKE, n=1 << 40):
    return ckv.lib.ckv_build_centroids_q8(R(cache or _q8()), labels, stride, T, None, R(graph or _graph()), ws, n, None)


BUILDS = [
    ("cache", lambda: _build(_q8(Hq=30)), INVALID),
    ("graph", lambda: _build(graph=_graph(S=-1)), INVALID),
    ("graph T_cap", lambda: _build(graph=_graph(T_cap=8192)), CAPACITY),
    ("labels", lambda: _build(labels=None), INVALID),
    ("T below S", lambda: _build(T=3), INVALID),
    ("T above T_cap", lambda: _build(T=4097, stride=5000), CAPACITY),
    ("labels stride", lambda: _build(stride=4095), INVALID),
    ("small ws", lambda: _build(n=1024), WORKSPACE),
    ("no ws", lambda: _build(ws=None), WORKSPACE),
]


@pytest.mark.parametrize("name,call,status", BUILDS, ids=[b[0] for b in BUILDS])
def test_build_refusals(name, call, status):
    assert call() == status, ckv.ckv_last_error()
    assert ckv.ckv_last_error()


@pytest.mark.parametrize("bad", [
    lambda c, g, lab, ws: ckv.ckv_build_centroids_q8(c, lab.long(), 8, g, ws),
    lambda c, g, lab, ws: ckv.ckv_build_centroids_q8(c, lab[:3], 8, g, ws),
    lambda c, g, lab, ws: ckv.ckv_build_centroids_q8(c, lab, 9, g, ws),
    lambda c, g, lab, ws: ckv.ckv_build_centroids_q8(c, lab.t().contiguous().t(), 8, g, ws),
    lambda c, g, lab, ws: ckv.ckv_build_centroids_q8(c, lab, 8, g, ws, torch.zeros(3, dtype=torch.int32)),
    lambda c, g, lab, ws: ckv.ckv_build_centroids_q8(c, lab, 8, g, ws, torch.zeros(2, dtype=torch.bool)),
    lambda c, g, lab, ws: ckv.ckv_build_centroids_q8(ckv.new_q8_cache(3, 2, 4, 64, 8, 16, 4, device="cpu"), lab, 8, g, ws),
    lambda c, g, lab, ws: ckv.ckv_build_centroids_q8(c, lab, 8, g, ws),  # not on a GPU
])
def test_build_binding_refuses(bad):
    c = ckv.new_q8_cache(2, 2, 4, 64, 8, 16, 4, device="cpu")
    g = ckv.new_graph(ckv.q8_shape(c, 64), ckv.PER_GROUP, 0, 4, 4, device="cpu")
    with pytest.raises(ValueError):
        bad(c, g, torch.zeros((4, 8), dtype=torch.int32), torch.zeros(1 << 16, dtype=torch.uint8))


@pytest.mark.parametrize("kw", [dict(tok_cap=0), dict(tok_cap=-5), dict(tok_cap=3), dict(tok_cap=1 << 30), dict(n_tok=None)])
def test_workspace_of_a_bad_selection_is_refused(kw):
    """A size for what no call would take (a negative capacity wrapped around) is not given out."""
    out = ctypes.c_size_t(77)
    st = ckv.lib.ckv_q8_workspace_size(R(_q8()), R(_graph()), R(_sel(**kw)), R(out))
    assert st == (3 if kw.get("tok_cap") == 1 << 30 else INVALID) and out.value == 77
    assert ckv.lib.ckv_q8_workspace_size(R(_q8()), None, R(_sel(**kw)), R(out)) == 0  # the dense call's alone


def test_the_error_word_is_read_on_its_own_device(monkeypatch):
    """With that device current, on its current stream; never through a host pointer."""
    cache = ckv.new_q8_cache(2, 2, 4, 64, 8, 16, 4, device="cpu")
    with pytest.raises(ValueError):
        ckv.ckv_get_device_error(cache)
    with pytest.raises(ValueError):
        ckv.ckv_get_device_error(ckv.new_graph(ckv.q8_shape(cache, 64), ckv.PER_GROUP, 0, 4, 4, device="cpu"))
    at = []

    class Word:
        device = torch.device("cuda", 3)

        def data_ptr(self):
            return FAKE

    class Table:
        desc, dev_err = ckv.TableDesc(), Word()

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            at.append(self.d)

        def __exit__(self, *a):
            at.append(None)

    class Lib:
        @staticmethod
        def ckv_get_device_error(desc, stream, code, reset):
            at.append(stream)
            return 0

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(ckv, "_stream", lambda s: ("stream of", at[-1], s))
    monkeypatch.setattr(ckv, "lib", Lib)
    assert ckv.ckv_get_device_error(Table()) == 0
    assert at == [torch.device("cuda", 3), ("stream of", torch.device("cuda", 3), None), None]


def test_trim_null_descriptors():
    assert ckv.lib.ckv_trim_graph_q8(None, R(_graph()), None) == INVALID
    assert ckv.lib.ckv_trim_graph_q8(R(_q8(_table())), None, None) == INVALID
    src = open(HEADER).read()
    assert int(re.search(r"#define CKV_DEVERR_CUT (\d+)", src).group(1)) == ckv.DEVERR_CUT


def test_binding_refuses_another_cachess_graph():
    a, b = (ckv.new_q8_cache(B, 2, 4, 64, 8, 16, 4, device="cpu") for B in (2, 3))
    graph = ckv.new_graph(ckv.q8_shape(b, 64), ckv.PER_GROUP, 0, 4, 4, device="cpu", undo=True)
    assert graph.undo.shape == (6, 4, 64) and graph.built.tolist() == [0] * 6
    assert ckv.new_graph(ckv.q8_shape(b, 64), ckv.PER_GROUP, 0, 4, 4, device="cpu").undo is None
    with pytest.raises(ValueError):
        ckv.ckv_trim_graph_q8(a, graph)
    with pytest.raises(ValueError):  # not on a GPU
        ckv.ckv_trim_graph_q8(b, graph)


# ---------------------------------------------------------------------------
# on the GPU
# ---------------------------------------------------------------------------

class Batch:
    """Requests of T tokens with communities, and decode steps over them."""

    def __init__(self, B=3, mode="group", T=90, d=64, dtype=torch.float32, fmt="int8", S=4, C=5, max_tail=8, n_blocks=60,
                 rule="score", seed=0):
        self.gen = torch.Generator().manual_seed(seed)
        self.Hkv, self.Hq, self.d, self.B, self.C, self.S = 2, 4, d, B, C, S
        self.cache = ckv.new_q8_cache(B, 2, 4, d, n_blocks, 16, 12, fmt, dtype)
        self.st = PagedLayerState(self.cache, mode, S, C, max_tail, T_cap=160, rule=rule)
        self.G = 2 if mode == "group" else 4
        self.mu = torch.randn((C, d), generator=self.gen)
        lab = torch.randint(0, C, (B, 2, T), generator=self.gen)
        K = self.mu[lab] + 0.3 * torch.randn((B, 2, T, d), generator=self.gen)
        V = torch.randn((B, 2, T, d), generator=self.gen)
        K, V = (x.to(dtype).to(DEV).transpose(1, 2) for x in (K, V))
        self.st.grow(i32([T] * B), B * T)
        self.st.write(K, V)
        self.labels = lab[:, :, None, :].expand(B, 2, self.G // 2, T).reshape(B * self.G, T).to(torch.int32).clone()
        self.labels[:, :S] = -1
        self.st.build(self.labels.to(DEV), T)

    def q(self):
        return torch.randn((self.B, 4, self.d), generator=self.gen).to(self.cache.dtype).to(DEV)

    def rows(self):
        k = self.mu[torch.randint(0, self.C, (self.B, 2), generator=self.gen)] + 0.3 * torch.randn((self.B, 2, self.d), generator=self.gen)
        v = torch.randn((self.B, 2, self.d), generator=self.gen)
        return tuple(x.to(self.cache.dtype).to(DEV) for x in (k, v))

    def join(self, k, q=None):
        q = self.q() if q is None else q
        self.st.select(q, 10 ** 6)
        return self.st.attend(q, k).clone()

    def step(self, add):
        """Attend and join, then grow by `add`; rows for every token added."""
        k, v = self.rows()
        out = self.join(k)
        p = self.st.grow(i32(add), self.B)
        live = [b for b, a in enumerate(add) if a > 0]
        pad = self.B - len(live)
        packed = [torch.cat([x[live], torch.zeros((pad, 2, self.d), dtype=x.dtype, device=DEV)]) for x in (k, v)]
        self.st.write(*packed)
        return p, out

    def state(self):
        g = self.st.graph
        s = {f: getattr(g, f).clone() for f in FIELDS}
        for f in ("tail_tok", "tail_comm"):
            s[f] = [getattr(g, f)[u, : int(g.tail_len[u])].tolist() for u in range(g.U)]
        return s

    def check_lists(self):
        """Every token that a community holds is listed once when all communities are selected."""
        self.st.select(self.q(), 10 ** 6)
        g, sel = self.st.graph, self.st.sel
        assert int(sel.n_sel.min()) >= 0
        for u in range(g.U):
            n = int(self.cache.len[u // self.G])
            got = sel.sel_tok[u, : int(sel.n_tok[u])].tolist()
            held = [t for t, c in enumerate(g.comm_of[u].tolist()) if c >= 0]
            assert sorted(got) == sorted(list(range(self.S)) + held), u
            assert len(set(got)) == len(got) and (not held or max(held) < n)
            assert int(g.cnt[u].sum()) == len(held)

    def errors(self):
        return ckv.ckv_get_device_error(self.cache, reset=True), ckv.ckv_get_device_error(self.st.graph, reset=True)


def same(a, b, rows=None):
    for f in a:
        x, y = a[f], b[f]
        if rows is not None:
            x, y = [x[u] for u in rows], [y[u] for u in rows]
            assert all(torch.equal(p, q) if torch.is_tensor(p) else p == q for p, q in zip(x, y)), f
        else:
            assert torch.equal(x, y) if torch.is_tensor(x) else x == y, f


KINDS = [dict(), dict(mode="head", d=128, dtype=torch.bfloat16), dict(fmt="e4m3", rule="vote"), dict(C=1, S=0, mode="head")]


@pytest.mark.gpu
@pytest.mark.parametrize("kw", KINDS)
def test_tokens_given_back_leave_their_communities(kw):
    b = Batch(**kw)
    b.step([1, 1, 1])
    before, lens = b.state(), b.cache.len.tolist()
    for _ in range(3):
        p, _ = b.step([1, 1, 1])
        assert p.granted.tolist() == [1, 1, 1]
    middle = b.state()
    assert b.st.graph.tail_len.tolist() == [4] * b.st.graph.U
    # request 0 keeps all, 1 loses two, 2 loses the three
    b.st.grow(i32([0, -2, -3]), 0)
    after = b.state()
    same(middle, after, range(b.G))
    same(before, after, range(2 * b.G, 3 * b.G))
    assert after["tail_len"].tolist() == [4] * b.G + [2] * b.G + [1] * b.G
    b.check_lists()
    # the same positions again, with other keys
    for _ in range(3):
        b.step([1, 1, 1])
        b.check_lists()
    assert b.cache.len.tolist() == [lens[0] + 6, lens[1] + 4, lens[2] + 3]
    b.st.grow(i32([-6, -4, -3]), 0)
    same(before, b.state())
    assert b.errors() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", KINDS)
def test_a_refused_or_idle_token_joins_nothing(kw):
    """Room for request 0 alone; request 2 adds nothing; the retry joins the position once."""
    T = 95
    b = Batch(T=T, n_blocks=3 * 6 + 1, **kw)
    b.step([1, 1, 0])  # 96 tokens: six whole blocks
    before = b.state()
    assert before["tail_len"].tolist() == [1] * b.G + [1] * b.G + [0] * b.G
    p, _ = b.step([1, 1, 0])
    assert p.granted.tolist() == [1, 0, 0]
    assert b.errors() == (ckv.DEVERR_PLAN, 0)
    same(before, b.state(), range(b.G, 3 * b.G))
    b.check_lists()
    b.st.grow(i32([-2, 0, 0]), 0)  # a block comes back
    p, _ = b.step([0, 1, 1])
    assert p.granted.tolist() == [0, 1, 1]
    b.check_lists()
    g = b.st.graph
    assert g.tail_tok[b.G: 2 * b.G, :2].tolist() == [[T, T + 1]] * b.G
    assert g.tail_tok[2 * b.G:, :1].tolist() == [[T]] * b.G
    assert g.tail_len.tolist() == [0] * b.G + [2] * b.G + [1] * b.G
    assert b.errors() == (0, 0)


@pytest.mark.gpu
def test_the_same_position_joined_again_replaces_the_first():
    """Two joins with no growth between them leave what the second alone would."""
    a, b = Batch(seed=5), Batch(seed=5)
    q = a.q()
    k1, k2 = a.rows()[0], a.rows()[0]
    a.st.select(q, 10 ** 6)
    a.st.attend(q, k1)
    a.st.attend(q, k2)
    b.st.select(q, 10 ** 6)
    b.st.attend(q, k2)
    same(a.state(), b.state())
    assert torch.equal(a.st.assigned, b.st.assigned) and a.st.graph.tail_len.tolist() == [1] * a.st.graph.U
    # a graph without room to undo does not join it a second time
    shape, ws = a.st.shape, a.st.graph_ws
    plain = ckv.new_graph(shape, ckv.PER_GROUP, a.S, a.C, 8)
    k, _ = a.st.read(90)
    rows = ckv.CacheDesc(shape.dtype, shape.B, shape.Hkv, shape.Hq, shape.d, shape.T_cap, k.data_ptr(), k.data_ptr(),
                         k.stride(0), k.stride(1), k.stride(2))
    ckv.ckv_build_centroids(rows, a.labels.to(DEV), 90, plain, ws)
    ckv.ckv_score_select(shape, plain, q, 10 ** 6, a.st.sel, ws)
    for i, key in enumerate((k1, k2)):
        ckv.ckv_sparse_decode_q8(a.cache, q, plain, a.st.sel, a.st.out, None, a.st.ws, key, a.st.assigned)
        assert (a.st.assigned >= 0).all() == (i == 0)
        assert plain.tail_len.tolist() == [1] * plain.U
    assert (a.st.assigned == -1).all() and int(plain.dev_err) == ckv.DEVERR_INDEX
    with pytest.raises(ckv.CKVError):
        ckv.ckv_trim_graph_q8(a.cache, plain)


@pytest.mark.gpu
def test_an_ended_request_loses_its_communities_and_no_other():
    b = Batch()
    b.step([1, 1, 1])
    before = b.state()
    b.st.grow(i32([0, -10 ** 6, 0]), 0)
    after = b.state()
    mine = range(b.G, 2 * b.G)
    same(before, after, [u for u in range(3 * b.G) if u not in mine])
    for u in mine:
        assert not after["cnt"][u].any() and not after["offs"][u].any() and (after["comm_of"][u] == -1).all()
        assert int(after["num_comm"][u]) == int(after["tail_len"][u]) == int(after["built"][u]) == 0
    assert b.errors() == (0, 0)  # an end is no fault
    b.st.select(b.q(), 10 ** 6)
    assert [int(b.st.sel.n_tok[u]) for u in mine] == [b.S] * b.G and [int(b.st.sel.n_sel[u]) for u in mine] == [0] * b.G
    # below the build's positions without an end: emptied, and said so
    b.st.grow(i32([-30, 0, 0]), 0)
    assert b.errors() == (0, ckv.DEVERR_CUT)
    same(before, b.state(), range(2 * b.G, 3 * b.G))
    assert int(b.st.graph.num_comm[: 2 * b.G].max()) == 0


@pytest.mark.gpu
def test_a_join_below_the_builds_positions_is_refused():
    """Lengths set behind the plan's back: the position is a member already."""
    b = Batch()
    before = b.state()
    b.cache.len[1] = 50
    b.join(b.rows()[0])
    after = b.state()
    same(before, after, range(b.G, 2 * b.G))
    assert b.st.assigned[b.G: 2 * b.G].tolist() == [-1] * b.G and int(b.st.assigned[: b.G].min()) >= 0
    assert b.errors()[1] == ckv.DEVERR_CUT
    b.cache.len[1] = 10 ** 6  # a bad length: nothing is done for this request
    b.cache.len[2] = -1
    ckv.ckv_trim_graph_q8(b.cache, b.st.graph)
    assert b.errors()[0] == ckv.DEVERR_BLOCK
    same(after, b.state(), range(b.G, 3 * b.G))


@pytest.mark.gpu
def test_full_tails_and_long_drops():
    """More joins than the tail holds, then all of them given back."""
    b = Batch(max_tail=3)
    before = b.state()
    for _ in range(5):
        b.step([1, 1, 1])
    assert b.st.graph.tail_len.tolist() == [3] * b.st.graph.U
    assert b.errors() == (0, ckv.DEVERR_TAIL_FULL)
    b.check_lists()
    b.st.grow(i32([-1, -3, -5]), 0)
    assert b.st.graph.tail_len.tolist() == [3] * b.G + [2] * b.G + [0] * b.G
    same(before, b.state(), range(2 * b.G, 3 * b.G))
    none = Batch(max_tail=0)
    before = none.state()
    none.step([1, 1, 1])
    none.st.grow(i32([-1, 0, 0]), 0)
    same(before, none.state())
    assert none.errors() == (0, ckv.DEVERR_TAIL_FULL)


@pytest.mark.gpu
def test_captured_steps_with_drops():
    """Two steps and a drop of one token, captured and replayed, against the same calls made eagerly."""
    a, b = Batch(seed=3), Batch(seed=3)
    q, (k, v) = a.q(), a.rows()
    one, back = i32([1, 1, 1]), i32([-1, 0, -1])

    def work(x):
        for add in (one, one):
            x.st.select(q, 60)
            x.st.attend(q, k)
            x.st.grow(add, 3)
            x.st.write(k, v)
        x.st.grow(back, 0)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(b)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work(b)
    work(a)
    for _ in range(2):
        work(a)
        g.replay()
        torch.cuda.synchronize()
        same(a.state(), b.state())
        assert torch.equal(a.st.out, b.st.out) and a.cache.len.tolist() == b.cache.len.tolist()
    b.check_lists()
    assert b.errors() == (0, 0)


@pytest.mark.gpu
def test_the_debug_build_trims_alike():
    b = Batch()
    before = b.state()
    b.step([1, 1, 1])
    b.cache.len.sub_(1)
    dbg = ckv.load_debug_library()
    assert dbg.ckv_trim_graph_q8(R(b.cache.desc), R(b.st.graph.desc), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    same(before, b.state())


@pytest.mark.gpu
def test_restored_centres_are_the_oracles():
    """After a drop the centres are the plain running means of what is left: the labelled values and the joined keys."""
    b = Batch(dtype=torch.float32)
    g = b.st.graph
    held, _ = b.st.read(90)
    joined = [{} for _ in range(g.U)]
    for i in range(4):
        k, v = b.rows()
        b.join(k)
        for u in range(g.U):
            joined[u][90 + i] = (int(b.st.assigned[u]), k[u // b.G, u % b.G].double().cpu().numpy())
        b.st.grow(i32([1, 1, 1]), 3)
        b.st.write(k, v)
    b.st.grow(i32([-1, -2, -3]), 0)
    for u in range(g.U):
        req, kv = u // b.G, u % b.G
        n = int(b.cache.len[req])
        keys = held[req, kv].double().cpu().numpy()
        for c in range(b.C):
            rows = [keys[t] for t in range(b.S, 90) if int(b.labels[u, t]) == c]
            rows += [x for t, (cc, x) in joined[u].items() if cc == c and t < n]
            assert int(g.cnt[u, c]) == len(rows)
            if rows:
                # the mean's own rounding, and at most four steps of it with three each (k - c, times 1/(n + 1), n >= 1;
                # plus c), each at most 2^-24 of the largest value: 13 of them
                err = np.abs(g.cent[u, c].double().cpu().numpy() - np.mean(rows, 0)).max()
                assert err <= 13 * 2.0 ** -24 * np.abs(rows).max()


# ---------------------------------------------------------------------------
# requests of different length
# ---------------------------------------------------------------------------

def ragged(lens, mode="group", fmt="int8", dtype=torch.float32, d=64, S=4, C=7, block=32, seed=0, T_cap=5024):
    """A cache of these lengths, filled in one growth, and labels for each request's own positions (behind them: any)."""
    gen = torch.Generator().manual_seed(seed)
    B, n = len(lens), sum(lens)
    cache = ckv.new_q8_cache(B, 2, 4, d, n // block + B + 4, block, 160, fmt, dtype)
    st = PagedLayerState(cache, mode, S, C, 8, T_cap=T_cap)
    st.grow(i32(lens), n)
    st.write(*((torch.randn((n, 2, d), generator=gen) * torch.exp2(torch.randint(-3, 3, (n, 1, 1), generator=gen).float()))
               .to(dtype).to(DEV) for _ in range(2)))
    U = st.graph.U
    labels = torch.randint(0, C, (U, max(lens)), generator=gen, dtype=torch.int32)
    for u in range(U):
        labels[u, :S] = -1
        labels[u, lens[u * B // U]:] = -9  # never looked at
    return st, labels


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["group", "head"])
@pytest.mark.parametrize("fmt,dtype,d", [("int8", torch.float32, 64), ("e4m3", torch.float32, 128), ("int8", torch.bfloat16, 128)])
def test_build_over_requests_of_different_length(mode, fmt, dtype, d):
    """Each request's graph is, bit for bit, what the wide cache's build makes of its own positions; the values held are
    fp32 whatever the rows' type."""
    lens = [300, 0, 5000, 3, 17, 4, 4097]
    st, labels = ragged(lens, mode, fmt, dtype, d)
    st.build(labels.to(DEV), max(lens))
    assert ckv.ckv_get_device_error(st.cache) == 0 and int(st.graph.dev_err) == 0
    c = st.cache
    f32 = ckv.q8_cache(c.k, c.v, c.k_scale, c.v_scale, c.table, c.len, 4, torch.float32)
    K, V = (torch.empty((len(lens), 2, 5024, d), device=DEV) for _ in range(2))
    ckv.ckv_q8_read(f32, K, V)
    g, G = st.graph, st.graph.U // len(lens)
    wide = ckv.cache_desc(K, V, 4)
    for b, n in enumerate(lens):
        ref = ckv.new_graph(wide, g.desc.mode, min(4, n), 7, 8)
        ws = ckv.new_workspace(ckv.ckv_workspace_size(wide, ref))
        own = torch.full(labels.shape, 0, dtype=torch.int32)
        own[:, : min(4, n)] = -1
        own[b * G: (b + 1) * G, :n] = labels[b * G: (b + 1) * G, :n]
        ckv.ckv_build_centroids(wide, own.to(DEV), n, ref, ws)
        rows = slice(b * G, (b + 1) * G)
        for f in ("comm_of", "offs", "cnt", "cent", "cent_q", "cent_qs", "num_comm", "tail_len", "built"):
            assert torch.equal(getattr(ref, f)[rows], getattr(g, f)[rows]), (b, f)
        m = max(n - 4, 0)
        assert torch.equal(ref.tok[rows, :m], g.tok[rows, :m])
    # every token but the sinks is selectable, and nothing else
    q = torch.randn((len(lens), 4, d), device=DEV).to(dtype)
    st.select(q, 10 ** 6)
    for u in range(g.U):
        n = lens[u // G]
        assert sorted(st.sel.sel_tok[u, : int(st.sel.n_tok[u])].tolist()) == list(range(max(n, 4)))


@pytest.mark.gpu
def test_build_of_some_requests_leaves_the_others():
    """A request ends, another takes its row and is built alone; the others decode on."""
    b = Batch()
    b.step([1, 1, 1])
    before = b.state()
    b.st.grow(i32([0, -10 ** 6, 0]), 0)
    n = 37
    b.st.grow(i32([0, n, 0]), n)
    gen = torch.Generator().manual_seed(9)
    rows = torch.randn((2, n, 2, b.d), generator=gen).to(DEV)
    b.st.write(rows[0], rows[1])
    labels = torch.full((b.st.graph.U, 64), 10 ** 6, dtype=torch.int32)
    mine = list(range(b.G, 2 * b.G))
    labels[mine, :n] = torch.randint(0, b.C, (b.G, n), generator=gen, dtype=torch.int32)
    labels[mine, : b.S] = -1
    b.st.build(labels.to(DEV), requests=i32([0, 5, 0]))
    same(before, b.state(), [u for u in range(3 * b.G) if u not in mine])
    assert b.st.graph.built.tolist() == [90] * b.G + [n] * b.G + [90] * b.G
    for _ in range(2):
        p, _ = b.step([1, 1, 1])
        assert p.granted.tolist() == [1, 1, 1]
        b.check_lists()
    assert int(b.st.assigned.min()) >= 0 and b.errors() == (0, 0)


@pytest.mark.gpu
def test_build_flags_what_it_cannot_use():
    lens = [100, 60, 80]
    st, labels = ragged(lens, block=16, T_cap=160)
    g, G, c = st.graph, 2, st.cache
    st.build(labels[:, :90].contiguous().to(DEV))  # request 0 is longer than its labels
    assert int(g.dev_err) == ckv.DEVERR_LABEL_RANGE and ckv.ckv_get_device_error(c) == 0
    assert g.built.tolist() == [90] * G + [60] * G + [80] * G and g.cnt.sum(1).tolist() == [86] * G + [56] * G + [76] * G
    g.dev_err.zero_()
    st.build(labels.to(DEV))
    whole = [x.clone() for x in (g.cnt, g.cent)]
    assert int(g.dev_err) == 0
    c.len[1] = -5
    c.table[2, 1] = 10 ** 6  # positions 16..31 of request 2
    st.build(labels.to(DEV))
    assert ckv.ckv_get_device_error(c, reset=True) == ckv.DEVERR_BLOCK and int(g.dev_err) == 0
    assert torch.equal(whole[0][:G], g.cnt[:G]) and torch.equal(whole[1][:G], g.cent[:G])
    assert not g.cnt[G: 2 * G].any() and g.built[G: 2 * G].tolist() == [0] * G
    k, _ = st.read(80)  # zeros at those positions
    assert ckv.ckv_get_device_error(c, reset=True) == ckv.DEVERR_BLOCK
    for u in range(2 * G, 3 * G):
        rows = k[2, u % 2].double().cpu()
        for cc in range(7):
            at = (labels[u, :80] == cc).nonzero().flatten()
            if len(at):  # one rounding of the mean
                assert (g.cent[u, cc].double().cpu() - rows[at].mean(0)).abs().max() <= 2.0 ** -24 * rows.abs().max()
    c.len[1] = 160 * 16 + 1
    st.build(labels.to(DEV), requests=i32([1, 0, 0]))  # requests left out are not looked at
    assert ckv.ckv_get_device_error(c) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["group", "head"])
def test_empty_and_short_requests_decode_beside_long_ones(mode):
    """Rows without a request, and requests shorter than the sinks: their lists name sinks that are not there, which is no
    fault.  Outputs are those of the dense call, which every request's list covers."""
    lens = [0, 3, 300, 1, 4, 0, 17]
    st, labels = ragged(lens, mode)
    st.build(labels.to(DEV))
    c, G = st.cache, st.graph.U // len(lens)
    q, k = torch.randn((7, 4, 64), device=DEV), torch.randn((7, 2, 64), device=DEV)
    live = i32([1 if n else 0 for n in lens])
    for step in range(3):
        st.select(q, 10 ** 6)
        sparse = st.attend(q, k).clone()
        dense = st.dense(q, torch.empty_like(sparse))
        assert not sparse[0].any() and not sparse[5].any()
        K, V = st.read(300)
        S = torch.einsum("bhd,bhtd->bht", q.abs(), K.abs().repeat_interleave(2, 1)).max() / 8
        assert (sparse - dense).abs().max() <= 2 * Q.attention_tol(float(S), 300, float(V.abs().max()))  # one bound each
        asg = st.assigned.view(7, G)
        assert (asg[[0, 1, 3, 5]] == -1).all() and (asg[[2, 6]] >= 0).all()  # nobody to join, in the short ones
        st.grow(live, 7)
        st.write(*[torch.zeros((7, 2, 64), device=DEV)] * 2)
        st.grow(-live, 0)  # (tokens that joined nobody are read by the dense call alone)
        assert c.len.tolist() == lens
        assert ckv.ckv_get_device_error(c, reset=True) == 0 and ckv.ckv_get_device_error(st.graph) == 0
    c.len[1] = -1  # a bad length is one
    st.attend(q)
    assert ckv.ckv_get_device_error(c) == ckv.DEVERR_BLOCK


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("padded", [False, True])
def test_rows_of_refused_requests_leave_the_pool(fmt, padded):
    """Of three requests that grow in one call two are refused, for want of blocks and of table; their rows change no code
    and no scale, and the third's only its own slots'."""
    c = ckv.new_q8_cache(4, 2, 2, 64, 12, 16, 5, fmt, torch.float32)
    p = ckv.new_plan(c, 200)
    ckv.ckv_plan_blocks(c, i32([40, 10, 30, 70]), p)
    gen = torch.Generator().manual_seed(2)
    rows = torch.randn((2, 200, 2, 64), generator=gen).to(DEV)
    ckv.ckv_quant_append(c, p, rows[0], rows[1])
    assert p.granted.tolist() == [40, 10, 30, 70]
    before = [x.clone() for x in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)]
    add = [30, 5, 50, 20]  # one block is free: 0 wants two; 1 grows inside its block; 2 wants three; 3 passes the table
    ckv.ckv_plan_blocks(c, i32(add), p)
    assert p.granted.tolist() == [0, 5, 0, 0] and ckv.ckv_get_device_error(c, reset=True) == ckv.DEVERR_PLAN
    big = 100 * torch.randn((2, 200, 2, 64), generator=gen).to(DEV)
    if padded:
        ckv.ckv_quant_append(c, p, *(x.view(4, 50, 2, 64) for x in big))
    else:
        ckv.ckv_quant_append(c, p, big[0], big[1])
    block = int(c.table[1, 0])
    for now, old in zip((c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale), before):
        others = [x for x in range(12) if x != block]
        assert torch.equal(now[others], old[others])
        assert not torch.equal(now[block], old[block])
        if now.dim() == 4:
            assert torch.equal(now[block, :, 15:], old[block, :, 15:])  # rows behind the last token
    assert ckv.ckv_get_device_error(c) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-1, 40, 2 ** 31 - 1])
def test_plan_flags_blocks_out_of_range(bad):
    """A block id that is none, in the table of a request that gives it back or in the free list, is flagged by the plan
    that meets it, rows or not; an id that is not met is not looked at."""
    for rows in (0, 5000):
        c = ckv.new_q8_cache(3, 1, 1, 64, 40, 16, 12)
        p = ckv.new_plan(c, 200)
        ckv.ckv_plan_blocks(c, i32([33, 64, 100]), p)
        assert ckv.ckv_get_device_error(c) == 0
        c.table[0, 2] = bad
        c.blocks.free_list[0] = bad
        p = ckv.new_plan(c, rows)
        ckv.ckv_plan_blocks(c, i32([0, -64, 0]), p)
        assert ckv.ckv_get_device_error(c) == 0
        ckv.ckv_plan_blocks(c, i32([-1, 0, 0]), p)
        assert ckv.ckv_get_device_error(c, reset=True) == ckv.DEVERR_BLOCK
        assert c.len.tolist() == [32, 0, 100]
    # taken from the free list: the 30th block from its top, by a request of its own
    c = ckv.new_q8_cache(2, 1, 1, 64, 40, 16, 40)
    c.blocks.free_list[39 - 30] = bad
    p = ckv.new_plan(c, 640)
    ckv.ckv_plan_blocks(c, i32([30 * 16, 0]), p)
    assert ckv.ckv_get_device_error(c) == 0
    ckv.ckv_plan_blocks(c, i32([0, 16]), p)
    assert ckv.ckv_get_device_error(c) == ckv.DEVERR_BLOCK
    assert p.slot.tolist()[:16] == [-1] * 16


@pytest.mark.gpu
def test_joins_by_the_wide_calls_are_undone_too():
    """ckv_assign_update, ckv_append_assign and ckv_sparse_decode_append on the paged graph (rows read back into a wide
    cache): what they join, the trim takes out."""
    b = Batch(T=90)
    st, c = b.st, b.cache
    K, V = (torch.zeros((3, 2, 160, 64), device=DEV) for _ in range(2))
    k, v = st.read(90)
    K[:, :, :90], V[:, :, :90] = k, v
    wide = ckv.cache_desc(K, V, 4)
    ws = ckv.new_workspace(ckv.ckv_workspace_size(wide, st.graph, st.sel))
    before = b.state()
    states = []
    for pos, how in ((90, "fused"), (91, "append"), (92, "update")):
        q, (kn, vn) = b.q(), b.rows()
        st.select(q, 10 ** 6)
        ckv.ckv_sparse_decode(wide, q, st.graph, st.sel, st.out, st.nbr8, ws)
        if how == "fused":
            ckv.ckv_sparse_decode_append(wide, q, st.graph, st.sel, st.out, st.nbr8, pos, kn, vn, st.assigned, ws)
        elif how == "append":
            ckv.ckv_append_assign(wide, st.graph, pos, kn, vn, st.nbr8, st.assigned)
        else:
            K[:, :, pos], V[:, :, pos] = kn, vn
            ckv.ckv_assign_update(wide, st.graph, pos, st.nbr8, st.assigned)
        states.append(b.state())
        assert (st.assigned >= 0).all() and st.graph.tail_len.tolist() == [pos - 89] * 6
    c.len.copy_(i32([92, 91, 90]))
    ckv.ckv_trim_graph_q8(c, st.graph)
    after = b.state()
    for r, want in enumerate((states[1], states[0], before)):
        same(want, after, range(2 * r, 2 * r + 2))
