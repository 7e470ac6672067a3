"""The 4-bit cache as a decode step uses it: q|k|v from packed weights, pages reserved, the new rows appended,
attention, the o projection; forks, truncation and compaction between steps; all of it captured in a HIP graph."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import synth
from oracle import kv4
from tests.gpu_util import bf16_as_f64, dev_bf16, host_bf16, say
from tests.kv4_util import attention_bounds, batch, bf16, bits, filled_cache

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a HIP GPU", allow_module_level=True)

import bitmask_spmv_amd as nm  # noqa: E402


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return bf16_as_f64(host_bf16(t))


def i32(*shape, fill=0):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


class Decoder:
    """Some layers of attention over one page table: packed q|k|v and o, a 4-bit cache each."""

    def __init__(self, seed, slots, Hq, H, D, ps, N, cols, layers=2, K=512):
        self.Hq, self.H, self.D, self.ps, self.K, self.layers = Hq, H, D, ps, K, layers
        pack = lambda R, C, *ids: nm.nm_prune_pack(  # noqa: E731
            synth.device_weights(R, C, 0, 80, R, C, seed, *ids), nm.nm_col_norm(synth.device_calib_acts(C, 0, 81, C, seed, *ids)), 2, 4)
        self.qkv = [[pack(h * D, K, layer, i) for i, h in enumerate((Hq, H, H))] for layer in range(layers)]
        self.o = [pack(K, Hq * D, layer, 9) for layer in range(layers)]
        self.cache = torch.zeros((layers, N, kv4.page_bytes(ps, H, D)), dtype=torch.uint8, device="cuda")
        self.table, self.kv_len, self.refs = i32(slots, cols, fill=-1), i32(slots), i32(N)
        self.moves, self.count, self.want = i32(slots, 2), i32(1), i32(slots)
        self.q_start = i32(slots + 1)
        self.ws = torch.empty(max(nm.nm_spmv_multi_workspace_bytes([Hq * D, H * D, H * D], K, slots),
                                  nm.nm_spmv_workspace_bytes(K, Hq * D, slots), 16), dtype=torch.uint8, device="cuda")
        self.aws = torch.empty(max(16, nm.nm_kv4_attention_workspace_bytes(slots, slots, Hq, H, D, 1, cols * ps)),
                               dtype=torch.uint8, device="cuda")
        self.pws = torch.empty(max(16, nm.nm_kv_pages_workspace_bytes(slots, slots, N, cols)), dtype=torch.uint8, device="cuda")
        rows = lambda h: torch.empty((slots, h * D), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.out = [rows(Hq), rows(H), rows(H)]
        self.att = torch.empty((slots, Hq, D), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros((slots, Hq), device="cuda")
        self.seen = None

    def book(self):
        return self.table, self.kv_len, self.refs, self.ps

    def resize(self):
        nm.nm_kv_resize(self.want, *self.book(), self.moves, self.count, workspace=self.pws)
        nm.nm_kv_copy_pages(self.cache, self.moves)

    def step(self, x):
        """One token of every slot (q_start says which have one): x bf16 [slots, K] -> x + o(attention), layer by layer."""
        for layer in range(self.layers):
            q, k, v = nm.nm_spmv_multi(self.qkv[layer], x, outs=self.out, workspace=self.ws)
            q, k, v = (t.unflatten(1, (-1, self.D)) for t in (q, k, v))
            where = self.table, self.kv_len, self.q_start
            nm.nm_kv4_append(k, v, self.cache[layer], *where, self.ps)
            self.att.zero_()
            nm.nm_kv4_attention(q, self.cache[layer], *where, self.H, self.ps, 1, out=self.att, lse=self.lse, workspace=self.aws)
            if self.seen is not None:
                self.seen(layer, q, k, v)
            x = x + nm.nm_spmv(*self.o[layer], self.att.flatten(1), workspace=self.ws)
        return x


class Mirror:
    """The plain definitions beside a Decoder, fed with its q, k and v."""

    def __init__(self, d):
        self.d = d
        self.table, self.kv_len, self.refs = (t.cpu().numpy().copy() for t in (d.table, d.kv_len, d.refs))
        self.cache = [c.cpu().numpy().copy() for c in d.cache]
        d.seen = self.look

    def moved(self, moves):
        for c in self.cache:
            for a, b in moves:
                if a >= 0:
                    c[b] = c[a]

    def same(self, what):
        torch.cuda.synchronize()
        for name, a, b in zip(("table", "kv_len", "refcount"), (self.d.table, self.d.kv_len, self.d.refs),
                              (self.table, self.kv_len, self.refs)):
            assert (a.cpu().numpy() == b).all(), f"{what}: {name}"
        used = np.nonzero(self.refs)[0]
        for c, w in zip(self.d.cache, self.cache):
            assert (c[dev(used)].cpu().numpy() == w[used]).all(), f"{what}: cache"

    def look(self, layer, q, k, v):
        d = self.d
        qs = d.q_start.cpu().numpy()
        n = int(qs[-1])
        kv4.append(self.cache[layer], f64(k), f64(v), self.table, self.kv_len, qs, d.ps)
        used = np.nonzero(self.refs)[0]  # the pages in use alone: the pool may be large
        local = np.where(self.table >= 0, np.searchsorted(used, self.table), -1)
        r = kv4.attention(f64(q), self.cache[layer][used], local, self.kv_len, qs, d.ps, d.H, d.D**-0.5, 0)
        bo, bl = attention_bounds({a: b[:n] for a, b in r.items()})
        assert (np.abs(f64(d.att)[:n] - r["out"][:n]) <= bo).all()
        lse, want = d.lse.cpu().numpy()[:n].astype(np.float64), r["lse"][:n]
        empty = np.isinf(want)
        assert (lse[empty] == -np.inf).all() and (np.abs(lse - np.where(empty, 0, want))[~empty] <= bl[~empty]).all()


def starts(flags):
    return dev(np.concatenate([[0], np.cumsum(flags)]).astype(np.int32))


@pytest.mark.parametrize("Hq,H,D,ps,N,cols", [(8, 2, 128, 64, 40, 12), (4, 4, 64, 128, 30, 40), (8, 2, 64, 64, 20000, 6)])
def test_decode_steps_with_forks_truncation_and_compaction(Hq, H, D, ps, N, cols):
    say("decode steps", Hq, H, D, ps, N, cols)
    slots = 6
    d = Decoder(1, slots, Hq, H, D, ps, N, cols)
    m = Mirror(d)

    def resize(want):
        d.want.copy_(dev(np.asarray(want, dtype=np.int32)))
        d.resize()
        moves, _ = kv4.resize(np.asarray(want, dtype=np.int32), m.table, m.kv_len, m.refs, ps)
        m.moved(moves)
        m.same("resize")

    def tokens(flags, n):
        for _ in range(n):
            resize(np.where(flags, m.kv_len + 1, -1))
            d.q_start.copy_(starts(flags))
            x = d.step(torch.randn((slots, d.K), device="cuda").to(torch.bfloat16))
            assert torch.isfinite(x).all()
            m.same("step")

    # lengths that put the next tokens on both sides of a page's end; one slot stays free
    resize([ps - 1, 3, 2 * ps - 2, 1, 0, 0])
    tokens(np.array([1, 1, 1, 1, 0, 0]), 3)
    # two copies of slot 2, one of slot 0 over slot 3; they share pages until they write
    pairs = np.array([[2, 4], [2, 5], [0, 3]], dtype=np.int32)
    moves, count = i32(3, 2), i32(1)
    nm.nm_kv_fork(dev(pairs[:, 0].copy()), dev(pairs[:, 1].copy()), *d.book(), moves, count, workspace=d.pws)
    nm.nm_kv_copy_pages(d.cache, moves)
    m.moved(kv4.fork(pairs[:, 0], pairs[:, 1], m.table, m.kv_len, m.refs, ps)[0])
    m.same("fork")
    tokens(np.array([1, 0, 1, 1, 1, 1]), 3)
    # back by a few tokens into a shared page, one slot freed, then on
    resize([ps - 4, 0, -1, ps - 3, -1, 2])
    tokens(np.array([1, 1, 0, 1, 1, 1]), 2)
    moves = i32(N // 2, 2)
    nm.nm_kv_compact(*d.book(), moves, count, workspace=d.pws)
    nm.nm_kv_copy_pages(d.cache, moves)
    m.moved(kv4.compact(m.table, m.kv_len, m.refs, ps, N // 2)[0])
    m.same("compact")
    tokens(np.array([1, 1, 1, 0, 1, 1]), 2)


# one launch to each operator; several launches, joined through the workspace, and pages past one workgroup's
@pytest.mark.parametrize("Hq,H,D,N,cols,first", [(8, 2, 128, 64, 12, 60), (8, 2, 64, 20000, 80, 3000)])
def test_a_captured_step_replays_as_the_eager_one(Hq, H, D, N, cols, first):
    say("captured step", Hq, H, D, N, cols)
    slots, ps = 5, 64
    a, b = (Decoder(3, slots, Hq, H, D, ps, N, cols) for _ in range(2))
    xs = [torch.randn((slots, a.K), device="cuda").to(torch.bfloat16) for _ in range(7)]
    x = torch.empty_like(xs[0])
    active = np.array([1, 1, 0, 1, 1])

    def whole_step(d, x):
        d.want.copy_(torch.where(d.flags, d.kv_len + 1, d.kv_len))
        d.resize()
        return d.step(x)

    lens = np.array([first, 1, ps, 2 * ps - 3, 0], dtype=np.int32)
    for d in (a, b):
        d.flags = dev(active.astype(bool))
        d.q_start.copy_(starts(active))
        g = torch.Generator(device="cuda").manual_seed(5)  # earlier tokens: any codes, ordinary scales
        d.cache.copy_(torch.randint(120, 128, d.cache.shape, generator=g, device="cuda", dtype=torch.uint8))
        d.want.copy_(dev(lens))
        d.resize()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a.step(xs[0])  # first calls outside the capture; the rows that it writes are written again
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    a.cache.copy_(b.cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = whole_step(a, x)
    torch.cuda.synchronize()
    for i, xi in enumerate(xs):
        if i == 4:  # one sequence ends, another begins: the graph reads all of it from the device
            for d in (a, b):
                d.flags.copy_(dev(np.array([1, 0, 1, 1, 1], dtype=bool)))
                d.q_start.copy_(starts([1, 0, 1, 1, 1]))
        want = whole_step(b, xi)
        torch.cuda.synchronize()
        x.copy_(xi)
        graph.replay()
        torch.cuda.synchronize()
        for name, u, w in (("y", y, want), ("att", a.att, b.att), ("lse", a.lse, b.lse), ("cache", a.cache, b.cache),
                           ("table", a.table, b.table), ("kv_len", a.kv_len, b.kv_len), ("refs", a.refs, b.refs),
                           ("moves", a.moves, b.moves), ("missing", a.count, b.count)):
            assert torch.equal(u.view(torch.uint8), w.view(torch.uint8)), f"replay {i}: {name}"


def test_captured_prompts_and_two_graphs_of_one_workspace():
    """A prompt batch and a long decode batch, each captured with the same workspace and replayed in turn."""
    say("two graphs")
    g = np.random.default_rng(8)
    H, Hq, D, ps = 2, 8, 128, 64
    cases = []
    need = 16
    for rows, lens in (([150, 3, 1], [400, 3, 2500]), ([1, 2, 1], [9000, 700, 5])):
        table, kv_len, q_start, N = batch(g, rows, lens, ps)
        T = sum(rows)
        cache = dev(filled_cache(g, N, ps, H, D))
        qs = [dev_bf16(bits(bf16(g.standard_normal((T, Hq, D))))) for _ in range(4)]
        need = max(need, nm.nm_kv4_attention_workspace_bytes(T, len(rows), Hq, H, D, max(rows), table.shape[1] * ps))
        cases.append([cache, dev(table), dev(kv_len), dev(q_start), max(rows), qs])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs = []
    s = torch.cuda.Stream()
    for cache, table, kv_len, q_start, most, qs in cases:
        q, out = qs[0].clone(), torch.empty_like(qs[0])
        lse = torch.empty(q.shape[:2], device="cuda")
        run = lambda q=q, out=out, lse=lse, c=cache, t=table, n=kv_len, b=q_start, m=most: nm.nm_kv4_attention(  # noqa: E731
            q, c, t, n, b, H, ps, m, out=out, lse=lse, workspace=ws)
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            run()
        graphs.append((graph, q, out, lse))
    for i in range(4):
        want = []
        for (cache, table, kv_len, q_start, most, qs), (_, q, _, _) in zip(cases, graphs):
            want.append(nm.nm_kv4_attention(qs[i], cache, table, kv_len, q_start, H, ps, most))
            q.copy_(qs[i])
        torch.cuda.synchronize()
        for graph, _, out, lse in graphs:
            out.fill_(7.0)
            lse.fill_(7.0)
        for graph, *_ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (_, _, out, lse), (wo, wl) in zip(graphs, want):
            assert torch.equal(out.view(torch.int16), wo.view(torch.int16)) and torch.equal(lse, wl)


@pytest.mark.parametrize("rows,lens", [([1, 1], [400, 30]), ([1, 1], [4000, 70]), ([150, 2], [300, 2])])
@pytest.mark.parametrize("D", [64, 128])
def test_a_query_that_is_not_finite_spoils_its_own_row_alone(rows, lens, D):
    say("not finite", rows, lens, D)
    g = np.random.default_rng(6)
    H, Hq, ps = 2, 8, 64
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    cache = filled_cache(g, N, ps, H, D)
    args = dev(cache), dev(table), dev(kv_len), dev(q_start), H, ps, max(rows)
    q = bf16(g.standard_normal((sum(rows), Hq, D)))
    r = kv4.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5, 0)
    bo, bl = attention_bounds(r)
    bad = dev_bf16(bits(q))
    spoilt = np.zeros((sum(rows), Hq), dtype=bool)
    for t, h, ch, x in ((0, 0, 0, float("nan")), (0, 5, D - 1, float("inf")), (sum(rows) - 1, 3, 33, float("-inf"))):
        bad[t, h, ch] = x
        spoilt[t, h] = True
    out, lse = nm.nm_kv4_attention(bad, *args)
    out, lse = f64(out), lse.cpu().numpy().astype(np.float64)
    assert np.isnan(out[spoilt]).all() and np.isnan(lse[spoilt]).all()
    assert (np.abs(out - r["out"])[~spoilt] <= bo[~spoilt]).all() and (np.abs(lse - r["lse"])[~spoilt] <= bl[~spoilt]).all()
    # no key at all: nothing to spoil
    none = torch.zeros_like(args[2])
    o3, l3 = nm.nm_kv4_attention(bad, args[0], args[1], none, *args[3:])
    assert (o3 == 0).all() and (l3 == float("-inf")).all()


def test_row_tiles_of_a_workgroup_each_over_long_contexts():
    """Enough row tiles that none is split between workgroups, up to 60 blocks each and a few without any."""
    say("whole tiles")
    g = np.random.default_rng(12)
    H, Hq, D, ps = 8, 16, 64, 256
    lens = [3840, 1, 64, 65, 0, 3000] + [int(n) for n in g.integers(1, 3840, size=14)]
    rows = [1, 1, 2, 1, 1, 0] + [1] * 14
    table, kv_len, q_start, N = batch(g, rows, lens, ps)
    assert nm.nm_kv4_attention_workspace_bytes(sum(rows), len(rows), Hq, H, D, 2, table.shape[1] * ps) == 0
    cache = filled_cache(g, N, ps, H, D)
    q = bf16(g.standard_normal((sum(rows), Hq, D)))
    for window in (0, 500):
        r = kv4.attention(q, cache, table, kv_len, q_start, ps, H, D**-0.5, window)
        bo, bl = attention_bounds(r)
        out, lse = nm.nm_kv4_attention(dev_bf16(bits(q)), dev(cache), dev(table), dev(kv_len), dev(q_start), H, ps, 2, window=window)
        lse, empty = lse.cpu().numpy().astype(np.float64), np.isinf(r["lse"])
        assert (np.abs(f64(out) - r["out"]) <= bo).all()
        assert (lse[empty] == -np.inf).all() and (np.abs(lse[~empty] - r["lse"][~empty]) <= bl[~empty]).all()


def test_infinities_and_nan_are_stored_as_the_largest_number():
    """6 * 2^125 with their sign; the rest of their 32 channels lose against that, the next 32 do not."""
    say("store not finite")
    x = torch.full((1, 1, 64), 0.75, dtype=torch.bfloat16, device="cuda")
    raw = [0x7F80, 0xFF80, 0x7FC0, 0xFFFF, 0x7F81]
    x.view(torch.int16)[0, 0, :5] = torch.tensor([r - 65536 if r > 32767 else r for r in raw], dtype=torch.int16)
    cache = torch.zeros((1, kv4.page_bytes(64, 1, 64)), dtype=torch.uint8, device="cuda")
    args = i32(1, 1), i32(1, fill=1), dev(np.array([0, 1], np.int32)), 64
    nm.nm_kv4_append(x, x, cache, *args)
    want = np.concatenate([6 * 2.0**125 * np.array([1, -1, 1, -1, 1]), np.zeros(27), np.full(32, 0.75)])
    for y in nm.nm_kv4_unpack(cache, *args, torch.empty_like(x), torch.empty_like(x)):
        assert (f64(y)[0, 0] == want).all()


def test_calls_on_a_stream_that_the_tensors_were_not_made_on():
    say("another stream")
    g = np.random.default_rng(1)
    table, kv_len, q_start, N = batch(g, [1, 70], [3000, 70], 64)
    c, t, n, b = dev(filled_cache(g, N, 64, 2, 64)), dev(table), dev(kv_len), dev(q_start)
    k = dev_bf16(bits(bf16(g.standard_normal((71, 2, 64)))))
    q = dev_bf16(bits(bf16(g.standard_normal((71, 8, 64)))))
    c2 = c.clone()
    nm.nm_kv4_append(k, k, c, t, n, b, 64)
    want = nm.nm_kv4_attention(q, c, t, n, b, 2, 64, 70)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        nm.nm_kv4_append(k, k, c2, t, n, b, 64)
        got = nm.nm_kv4_attention(q, c2, t, n, b, 2, 64, 70)
    torch.cuda.synchronize()
    assert torch.equal(c, c2) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_arguments_that_are_refused():
    say("refused")
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    c = torch.zeros((4, kv4.page_bytes(64, 2, 64)), dtype=torch.uint8, device="cuda")
    t, n, b = i32(1, 2), i32(1), dev(np.array([0, 3], np.int32))
    ok = dict(k=x, v=x, cache=c, page_table=t, kv_len=n, q_start=b, page_size=64)
    for bad, err in ((dict(k=x.float()), TypeError), (dict(v=x[:2]), ValueError), (dict(k=x.cpu()), ValueError),
                     (dict(v=x.cpu()), ValueError), (dict(k=x[..., :32], v=x[..., :32]), ValueError), (dict(cache=c[:, :-16]), ValueError),
                     (dict(cache=c.view(torch.int8)), TypeError), (dict(page_table=t.long()), TypeError),
                     (dict(page_table=t[0]), ValueError), (dict(kv_len=i32(2)), ValueError), (dict(q_start=n), ValueError),
                     (dict(kv_len=n.cpu()), TypeError), (dict(page_size=128), ValueError),
                     (dict(k=x[:, :, ::2], v=x[:, :, ::2]), ValueError)):
        with pytest.raises(err):
            nm.nm_kv4_append(**{**ok, **bad})
    at = dict(q=x, cache=c, page_table=t, kv_len=n, q_start=b, n_kv=2, page_size=64, max_q_len=3)
    for bad, err in ((dict(q=x[:, :1]), RuntimeError), (dict(max_q_len=0), RuntimeError), (dict(window=-1), RuntimeError),
                     (dict(scale=float("nan")), RuntimeError), (dict(n_kv=1), ValueError), (dict(out=x.float()), TypeError),
                     (dict(lse=torch.zeros((3, 2), device="cuda", dtype=torch.float64)), ValueError),
                     (dict(page_table=i32(1, 40), workspace=c[0, :64]), RuntimeError)):
        with pytest.raises(err):
            nm.nm_kv4_attention(**{**at, **bad})
    m, one = i32(1, 2), i32(1)
    rs = dict(new_len=n, page_table=t, kv_len=n, refcount=i32(4), page_size=64, moves=m, missing=one)
    for bad, err in ((dict(moves=i32(2, 2)), ValueError), (dict(new_len=n.long()), TypeError), (dict(page_size=60), RuntimeError),
                     (dict(refcount=i32(2, 2)), ValueError)):
        with pytest.raises(err):
            nm.nm_kv_resize(**{**rs, **bad})
    with pytest.raises(ValueError):
        nm.nm_kv_copy_pages(c[:, :16], m)
    assert int(c.sum()) == 0
