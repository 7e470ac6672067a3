"""The 8-bit cache as a decode step uses it: rotated tokens in, blocks chosen, attention, pages that grow, are shared and move; captured in
a graph, on other streams, in caches larger than 4 GiB; and what is refused."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv4, kv8
from tests.gpu_util import bf16_as_f64, dev_bf16, host_bf16, say
from tests.kv4_util import batch, bf16, bits
from tests.kv8_util import filled_cache, turns

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a HIP GPU", allow_module_level=True)

import bitmask_spmv_amd as nm  # noqa: E402
from tests.test_gpu_kv8 import dev, held_to, same_bytes  # noqa: E402

H, HQ, D, PS = 2, 8, 128, 64


def rows(g, T, heads, size=1.0):
    return bf16(size * g.standard_normal((T, heads, D)))


def test_sequences_that_grow_fork_and_end():
    """Twelve steps of three slots against the oracle, step by step: prompts, single tokens, a fork, an end, drafts taken back."""
    say("steps")
    g = np.random.default_rng(0)
    S, N, cols = 3, 20, 8
    table, kv_len, refs = np.full((S, cols), -1, dtype=np.int32), np.zeros(S, dtype=np.int32), np.zeros(N, dtype=np.int32)
    cache = g.integers(0, 256, size=(N, kv8.page_bytes(PS, H, D)), dtype=np.uint8)
    turn = turns(g, cols * PS, D)
    td, ld, rd, cd, turn_d = dev(table), dev(kv_len), dev(refs), dev(cache), dev(turn)
    moves, missing = torch.full((S, 2), -1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    #            new rows of each slot, and what is done before
    steps = [([70, 0, 0], None), ([1, 130, 0], None), ([1, 1, 0], (0, 2)), ([1, 1, 1], None), ([5, 1, 1], None), ([-3, 1, 1], None),
             ([2, 1, 60], None), ([1, 1, 1], None), ([-200, 40, 1], None), ([33, 1, 8], None), ([1, 1, 9], (1, 0)), ([1, 1, 1], None)]
    for n, (grow, pair) in enumerate(steps):
        if pair:
            p, c = (np.array([x], dtype=np.int32) for x in pair)
            m = torch.full((1, 2), -1, dtype=torch.int32, device="cuda")
            nm.nm_kv_fork(dev(p), dev(c), td, ld, rd, PS, m, missing)
            want, lack = kv4.fork(p, c, table, kv_len, refs, PS)
            nm.nm_kv_copy_pages(cd, m)
            for a, b in want:
                if a >= 0:
                    cache[b] = cache[a]
            assert lack == 0 and (m.cpu().numpy() == want).all()
        new_len = np.maximum(kv_len + np.array(grow, dtype=np.int32), 0)
        nm.nm_kv_resize(dev(new_len), td, ld, rd, PS, moves, missing)
        want, lack = kv4.resize(new_len, table, kv_len, refs, PS)
        nm.nm_kv_copy_pages(cd, moves)
        for a, b in want:
            if a >= 0:
                cache[b] = cache[a]
        assert lack == 0 and (td.cpu().numpy() == table).all() and (ld.cpu().numpy() == kv_len).all()
        counts = [max(x, 0) for x in grow]
        q_start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        T = int(q_start[-1])
        k, v, q = rows(g, T, H, 1.0 + n % 3), rows(g, T, H), rows(g, T, HQ)
        args = cd, td, ld, dev(q_start)
        qr = nm.nm_kv8_append(dev_bf16(bits(k)), dev_bf16(bits(v)), *args, PS, rotation=turn_d, q=dev_bf16(bits(q)))
        kv8.append(cache, k, v, table, kv_len, q_start, PS, turn)
        same_bytes(cd, cache, PS, H, D, f"step {n}")
        q = bf16_as_f64(host_bf16(qr))
        sel = nm.nm_kv8_select(qr, *args, H, PS, 3, first=1, last=1)
        assert (sel.cpu().numpy() == kv8.select(q, cache, table, kv_len, q_start, PS, H, 3, 1, 1)).all()
        for s in (None, sel):
            out, lse = nm.nm_kv8_attention(qr, *args, H, PS, max(counts), selected=s)
            r = kv8.attention(q, cache, table, kv_len, q_start, PS, H, D**-0.5, 0, None if s is None else s.cpu().numpy())
            held_to(bf16_as_f64(host_bf16(out)), lse.cpu().numpy().astype(np.float64), r, f"step {n}")


def test_a_layer_of_packed_weights():
    """q|k|v of a pruned layer, rotation and append, choice, attention, o: four tokens of three slots, each step of it checked."""
    say("layer")
    import synth

    g = np.random.default_rng(1)
    slots, K, cols = 3, 512, 4
    pack = lambda R, C, i: nm.nm_prune_pack(  # noqa: E731
        synth.device_weights(R, C, 0, 80, R, C, i), nm.nm_col_norm(synth.device_calib_acts(C, 0, 81, C, i)), 2, 4)
    qkv, o = [pack(h * D, K, i) for i, h in enumerate((HQ, H, H))], pack(K, HQ * D, 9)
    start = np.array([130, 63, 0], dtype=np.int32)
    table, _, _, N = batch(g, [0] * slots, list(start + 4), PS, extra_cols=0)
    cols = table.shape[1]
    cache = filled_cache(g, N, PS, H, D)
    cd, td, turn = dev(cache), dev(table), turns(g, cols * PS, D)
    x = dev_bf16(bits(g.standard_normal((slots, K))))
    q_start = np.arange(slots + 1, dtype=np.int32)
    for step in range(4):
        kv_len = (start + step + 1).astype(np.int32)
        q, k, v = (t.unflatten(1, (-1, D)) for t in nm.nm_spmv_multi(qkv, x))
        k0, v0, q0 = (bf16_as_f64(host_bf16(t)) for t in (k, v, q))
        args = cd, td, dev(kv_len), dev(q_start)
        nm.nm_kv8_append(k, v, *args, PS, rotation=dev(turn), q=q, q_out=q)
        kv8.append(cache, k0, v0, table, kv_len, q_start, PS, turn)
        same_bytes(cd, cache, PS, H, D, f"step {step}")
        sel = nm.nm_kv8_select(q, *args, H, PS, 2)
        out, lse = nm.nm_kv8_attention(q, *args, H, PS, 1, selected=sel)
        qr = bf16_as_f64(host_bf16(q))
        assert np.abs(qr - np.stack([kv8.rotate(q0[s], kv_len[s] - 1, turn, False) for s in range(slots)])).max() <= 2.0**-7 * np.abs(q0).max()
        r = kv8.attention(qr, cache, table, kv_len, q_start, PS, H, D**-0.5, 0, sel.cpu().numpy())
        held_to(bf16_as_f64(host_bf16(out)), lse.cpu().numpy().astype(np.float64), r, f"step {step}")
        x = x + nm.nm_spmv(*o, out.flatten(1))
    assert torch.isfinite(x).all()


@pytest.mark.parametrize("rows_,lens,ps,top", [([1, 1, 1], [500, 64, 1], 64, 4), ([1], [20000], 512, 20), ([40, 3, 0], [30000, 900, 5], 512, 9),
                                               ([1, 1], [200000, 140000], 512, 16), ([500, 200], [700, 900], 64, 6)])
def test_a_captured_step_is_the_eager_one_at_every_replay(rows_, lens, ps, top):
    """Append, choice and attention (all keys, and chosen blocks) in one graph; lengths, queries and tokens change between replays."""
    say("graph", rows_, lens)
    g = np.random.default_rng(sum(rows_))
    table, kv_len, q_start, N = batch(g, rows_, lens, ps)
    T = int(q_start[-1])
    turn = dev(turns(g, table.shape[1] * ps, D))
    first = filled_cache(g, N, ps, H, D)
    k, v, q = (dev_bf16(bits(rows(g, T, h))) for h in (H, H, HQ))
    cache, td, ld, qd = dev(first), dev(table), dev(kv_len), dev(q_start)
    made = {}

    def step():
        made["q"] = nm.nm_kv8_append(k, v, cache, td, ld, qd, ps, rotation=turn, q=q)
        made["sel"] = nm.nm_kv8_select(made["q"], cache, td, ld, qd, H, ps, top, first=1, last=1)
        made["all"] = nm.nm_kv8_attention(made["q"], cache, td, ld, qd, H, ps, max(rows_))
        made["some"] = nm.nm_kv8_attention(made["q"], cache, td, ld, qd, H, ps, max(rows_), selected=made["sel"])

    step()  # the first launch of a kernel loads it
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    captured = dict(made)
    for replay in range(4):
        less = replay % 3
        shorter = np.maximum(kv_len - less, np.minimum(kv_len, np.array(rows_)))
        for to, h in ((k, H), (v, H), (q, HQ)):
            to.copy_(dev_bf16(bits(rows(g, T, h))))
        ld.copy_(dev(shorter.astype(np.int32)))
        cache.copy_(dev(first))
        graph.replay()
        torch.cuda.synchronize()
        got = [captured["q"].clone(), captured["sel"].clone(), *(x.clone() for x in captured["all"] + captured["some"]), cache.clone()]
        cache.copy_(dev(first))
        step()
        torch.cuda.synchronize()
        for name, a, b in zip(("q", "sel", "out", "lse", "some", "some lse", "cache"), got, [made["q"], made["sel"], *made["all"], *made["some"], cache]):
            assert torch.equal(a, b), f"replay {replay}: {name}"


def test_two_streams_at_once():
    """Calls that overlap in time, each with what it allocates, give what they give alone."""
    say("streams")
    g = np.random.default_rng(5)
    cases = []
    for lens in ([9000, 40, 3000], [5000, 8000, 1]):
        table, kv_len, q_start, N = batch(g, [1, 1, 1], lens, PS)
        cases.append((dev_bf16(bits(rows(g, 3, HQ))), dev(filled_cache(g, N, PS, H, D)), dev(table), dev(kv_len), dev(q_start)))

    def run(c):
        sel = nm.nm_kv8_select(*c, H, PS, 16, first=1, last=2)
        return (sel, *nm.nm_kv8_attention(*c, H, PS, 1, selected=sel), *nm.nm_kv8_attention(*c, H, PS, 1))
    alone = [run(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for c, st in zip(cases, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(run(c))
        for st in streams:
            st.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_pages_behind_four_gibibytes():
    say("large cache")
    g = np.random.default_rng(6)
    N = (1 << 32) // kv8.page_bytes(PS, H, D) + 40
    lens, rows_ = [300, 200], [2, 150]
    table, kv_len, q_start, n = batch(g, rows_, lens, PS)
    high = np.where(table >= 0, table + N - n, -1).astype(np.int32)
    small = filled_cache(g, n, PS, H, D)
    cache = torch.zeros((N, small.shape[1]), dtype=torch.uint8, device="cuda")
    cache[N - n :] = dev(small)
    T = int(q_start[-1])
    k, v, q = rows(g, T, H), rows(g, T, H), rows(g, T, HQ)
    args = dev(high), dev(kv_len), dev(q_start)
    nm.nm_kv8_append(dev_bf16(bits(k)), dev_bf16(bits(v)), cache, *args, PS)
    kv8.append(small, k, v, table, kv_len, q_start, PS)
    same_bytes(cache[N - n :], small, PS, H, D, "large cache")
    qd = dev_bf16(bits(q))
    sel = nm.nm_kv8_select(qd, cache, *args, H, PS, 2, first=0, last=1)
    assert (sel.cpu().numpy() == kv8.select(q, small, table, kv_len, q_start, PS, H, 2, 0, 1)).all()
    out, lse = nm.nm_kv8_attention(qd, cache, *args, H, PS, 150)
    r = kv8.attention(q, small, table, kv_len, q_start, PS, H, D**-0.5)
    held_to(bf16_as_f64(host_bf16(out)), lse.cpu().numpy().astype(np.float64), r, "large cache")
    ko, vo = torch.empty_like(qd[:, :H]), torch.empty_like(qd[:, :H])
    nm.nm_kv8_unpack(cache, *args, PS, ko.contiguous(), vo.contiguous())


def test_results_are_the_same_every_time():
    say("again")
    g = np.random.default_rng(7)
    lens = [int(n) for n in g.integers(1, 9000, 20)]
    table, kv_len, q_start, N = batch(g, [1] * 20, lens, PS)
    c = dev_bf16(bits(rows(g, 20, HQ))), dev(filled_cache(g, N, PS, H, D)), dev(table), dev(kv_len), dev(q_start)
    a = nm.nm_kv8_select(*c, H, PS, 24, first=1, last=2), *nm.nm_kv8_attention(*c, H, PS, 1)
    for _ in range(10):
        b = nm.nm_kv8_select(*c, H, PS, 24, first=1, last=2), *nm.nm_kv8_attention(*c, H, PS, 1)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_no_rows_and_no_sequences():
    say("nothing")
    z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    i32 = torch.int32
    cache = z(2, kv8.page_bytes(PS, H, D), dtype=torch.uint8)
    for S in (0, 3):
        args = cache, z(S, 2, dtype=i32), z(S, dtype=i32), z(S + 1, dtype=i32)
        nm.nm_kv8_append(z(0, H, D), z(0, H, D), *args, PS)
        nm.nm_kv8_unpack(*args, PS, z(0, H, D), z(0, H, D))
        assert nm.nm_kv8_select(z(0, HQ, D), *args, H, PS, 4).shape == (0, H, 4)
        assert nm.nm_kv8_attention(z(0, HQ, D), *args, H, PS, 1)[0].shape == (0, HQ, D)
    assert (cache == 0).all()


def test_refusals():
    """Every one before anything is launched."""
    say("refusals")
    z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    i32, u8 = torch.int32, torch.uint8
    T, S, cols = 3, 2, 4
    k, q = z(T, H, D), z(T, HQ, D)
    ok = [z(5, kv8.page_bytes(PS, H, D), dtype=u8), z(S, cols, dtype=i32), z(S, dtype=i32), z(S + 1, dtype=i32)]
    turn = z(cols * PS, D // 2, 2, dtype=torch.float32)
    bad_batches = [
        [z(5, kv4.page_bytes(PS, H, D), dtype=u8), *ok[1:]], [ok[0].to(torch.int8), *ok[1:]], [ok[0][:, :-128], *ok[1:]],
        [ok[0], ok[1].long(), *ok[2:]], [ok[0], ok[1].t(), *ok[2:]], [*ok[:2], z(S + 1, dtype=i32), ok[3]], [*ok[:3], z(S, dtype=i32)],
        [*ok[:2], ok[2].cpu(), ok[3]]]
    errors = (ValueError, TypeError, nm.NmError)
    for b in bad_batches:
        with pytest.raises(errors):
            nm.nm_kv8_append(k, k, *b, PS)
        with pytest.raises(errors):
            nm.nm_kv8_unpack(*b, PS, k, k)
        with pytest.raises(errors):
            nm.nm_kv8_select(q, *b, H, PS, 4)
        with pytest.raises(errors):
            nm.nm_kv8_attention(q, *b, H, PS, 1)
    for kw in (dict(rotation=turn.double()), dict(rotation=turn[:-1]), dict(rotation=turn[..., 0]), dict(rotation=turn[:, :12]), dict(rotation=turn.cpu()),
               dict(rotation=turn[:, ::2]), dict(q=q), dict(q_out=q), dict(rotation=turn, q=q[:2]), dict(rotation=turn, q=q.float()),
               dict(rotation=turn, q=q, q_out=q[:, :4]), dict(rotation=turn, q=z(T, 3, D)), dict(rotation=turn, q=q.cpu())):
        with pytest.raises(errors):
            nm.nm_kv8_append(k, k, *ok, PS, **kw)
    with pytest.raises(errors):
        nm.nm_kv8_append(k, k[:, :1], *ok, PS)
    with pytest.raises(errors):
        nm.nm_kv8_append(k.float(), k, *ok, PS)
    for top, kw in ((0, {}), (1, dict(first=1, last=1)), (4, dict(first=-1)), (4, dict(out=z(T, H, 5, dtype=i32))), (4, dict(out=z(T, H, 4))),
                    (4, dict(out=z(T, H + 1, 4, dtype=i32))), (4, dict(out=z(H, T, 4, dtype=i32).transpose(0, 1)))):
        with pytest.raises(errors):
            nm.nm_kv8_select(q, *ok, H, PS, top, **kw)
    sel = z(T, H, 4, dtype=i32)
    for kw in (dict(scale=float("nan")), dict(scale=1e30), dict(window=-1), dict(selected=sel.long()), dict(selected=sel[:2]), dict(selected=sel[..., :0]),
               dict(selected=sel[..., ::2]), dict(selected=sel.cpu()), dict(out=q[:, :4]), dict(lse=z(T, HQ)), dict(workspace=z(8, dtype=u8), max_q_len=0)):
        with pytest.raises(errors):
            nm.nm_kv8_attention(q, *ok, H, PS, kw.pop("max_q_len", 1), **kw)
    with pytest.raises(errors):
        nm.nm_kv8_attention(q[:, :3], *ok, H, PS, 1)
    long = [ok[0], z(S, 400, dtype=i32), *ok[2:]]
    with pytest.raises(nm.NmError, match="WORKSPACE"):
        nm.nm_kv8_attention(q, *long, H, PS, 1, workspace=z(64, dtype=u8))
    with pytest.raises(nm.NmError, match="WORKSPACE"):
        nm.nm_kv8_select(q[:2].repeat(1, 1, 1), ok[0], z(S, 3000, dtype=i32), *ok[2:], H, PS, 4, workspace=z(64, dtype=u8))
