"""Page keeping on the GPU against the plain definitions (oracle/kv4.py), number for number."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv4
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a HIP GPU", allow_module_level=True)

import bitmask_spmv_amd as nm  # noqa: E402


class Pool:
    """Tables on both sides: the GPU's and the plain ones."""

    def __init__(self, seed, S, cols, N, ps, lens):
        self.g = np.random.default_rng(seed)
        self.ps = ps
        self.table, self.kv_len, self.refs = np.full((S, cols), -1, np.int32), np.zeros(S, np.int32), np.zeros(N, np.int32)
        order, at = self.g.permutation(N), 0
        for s, n in enumerate(lens):
            c = -(-n // ps)
            self.table[s, :c], self.kv_len[s] = order[at : at + c], n
            self.refs[order[at : at + c]] = 1
            at += c
        self.d = [torch.from_numpy(a.copy()).cuda() for a in (self.table, self.kv_len, self.refs)]

    def same(self, what, moves, count, md, cd):
        torch.cuda.synchronize()
        for name, a, b in zip(("table", "kv_len", "refcount"), self.d, (self.table, self.kv_len, self.refs)):
            assert (a.cpu().numpy() == b).all(), f"{what}: {name}"
        assert (md.cpu().numpy() == moves).all(), f"{what}: moves"
        assert int(cd) == count, f"{what}: count"

    def out(self, n):
        return torch.full((n, 2), 99, dtype=torch.int32, device="cuda"), torch.full((1,), 99, dtype=torch.int32, device="cuda")

    def resize(self, new):
        new = np.asarray(new, dtype=np.int32)
        md, cd = self.out(len(new))
        nm.nm_kv_resize(torch.from_numpy(new).cuda(), *self.d, self.ps, md, cd)
        self.same("resize", *kv4.resize(new, self.table, self.kv_len, self.refs, self.ps), md, cd)
        return md

    def fork(self, parent, child):
        p, c = np.asarray(parent, dtype=np.int32), np.asarray(child, dtype=np.int32)
        md, cd = self.out(len(p))
        nm.nm_kv_fork(torch.from_numpy(p).cuda(), torch.from_numpy(c).cuda(), *self.d, self.ps, md, cd)
        self.same("fork", *kv4.fork(p, c, self.table, self.kv_len, self.refs, self.ps), md, cd)
        return md

    def compact(self, most):
        md, cd = self.out(most)
        nm.nm_kv_compact(*self.d, self.ps, md, cd)
        self.same("compact", *kv4.compact(self.table, self.kv_len, self.refs, self.ps, most), md, cd)
        return md


@pytest.mark.parametrize("N,S,ps", [(10, 4, 64), (64, 9, 128), (4096, 40, 64), (4097, 300, 64), (16384, 1024, 64), (16384, 256, 64), (5000, 190, 256),
                                    (16385, 30, 64), (20000, 700, 512), (40000, 1100, 128)])
def test_a_long_run_of_operators(N, S, ps):
    """Random growth, truncation, forks (some of them refused) and compaction, the pool short at times."""
    say("pool", N, S, ps)
    cols = max(2, 2 * N // S)
    g = np.random.default_rng(N)
    p = Pool(N, S, cols, N, ps, [int(g.integers(0, max(1, N // (2 * S)) * ps + 1)) for _ in range(S)])
    for step in range(12):
        kind = step % 4
        if kind == 0:
            new = p.kv_len + g.integers(0, 2 * ps, size=S)
            new[g.random(S) < 0.2] = -1
            p.resize(new)
        elif kind == 1:
            n = max(1, S // 3)
            p.fork(g.integers(-1, S + 1, size=n), g.integers(-1, S + 1, size=n))
        elif kind == 2:
            new = (p.kv_len * g.random(S)).astype(np.int64) + g.integers(0, 3, size=S) * (g.random(S) < 0.5)
            new[g.random(S) < 0.3] = 0
            p.resize(new)
        else:
            p.compact(int(g.integers(1, N // 2 + 2)))
        assert (p.refs >= 0).all()
        held = p.table[p.table >= 0]
        assert (np.bincount(held, minlength=N) == p.refs).all()


def test_the_same_pair_and_chains_are_refused():
    say("refused pairs")
    p = Pool(1, 8, 4, 40, 64, [100, 64, 30, 0, 200, 0, 0, 7])
    p.fork([0, 0, 3, 4, 1, 2, 0], [5, 5, 6, 4, 8, -1, 3])  # slot 5 twice; parent 3 is a child; itself; no slot
    p.fork([0, 0, 0, 1], [6, 7, 2, 3])  # children that held pages


def test_two_that_share_a_partial_page_and_both_grow():
    say("shared tails")
    p = Pool(2, 4, 4, 12, 64, [100, 0, 0, 64])
    p.table[1], p.kv_len[1] = p.table[0], 100  # as a program that truncates into a shared page leaves it
    p.refs[p.table[0, :2]] += 1
    p.d = [torch.from_numpy(a.copy()).cuda() for a in (p.table, p.kv_len, p.refs)]
    p.resize([101, 190, 1, 64])
    p.resize([-1, 128, 64, 65])
    p.resize([128 * 3, 1, 0, 64])  # more than four columns: left alone


def test_nothing_to_do_and_a_full_pool():
    say("full pool")
    p = Pool(3, 3, 4, 5, 64, [64, 100, 128])
    p.resize([64, 100, 128])
    p.resize([65, 129, 129])
    p.fork([1], [0])  # the child's own page is free again before its copy is asked for
    p.fork([2], [1])
    p.resize([0, 0, 0])
    p.compact(3)
    p.resize([256, 1, 1])


@pytest.mark.parametrize("layers,N,nbytes", [(1, 5, 16), (1, 9, 4352), (3, 7, 69632), (2, 300, 16400), (1, 3, 1 << 20)])
def test_copy_pages(layers, N, nbytes):
    say("copy", layers, N, nbytes)
    g = np.random.default_rng(N)
    whole = torch.from_numpy(g.integers(0, 256, size=(layers, N + 1, nbytes), dtype=np.uint8)).cuda()
    cache = whole[:, :N]  # a layer stride of its own
    want = cache.clone()
    perm = g.permutation(N)
    k = N // 2
    moves = np.concatenate([np.stack([perm[g.integers(0, k, size=N - k)], perm[k:]], 1),
                            [[-1, -1], [0, -1], [N, 0], [0, N], [2, 2], [-5, 1]]]).astype(np.int32)
    for a, b in moves[: N - k]:
        want[:, b] = cache[:, a]
    last = whole[:, N].clone()
    if layers == 1:
        cache = cache[0]
    nm.nm_kv_copy_pages(cache, torch.from_numpy(moves).cuda())
    assert torch.equal(whole[:, :N], want) and torch.equal(whole[:, N], last)


def test_an_empty_list_of_moves():
    cache = torch.zeros((2, 16), dtype=torch.uint8, device="cuda")
    nm.nm_kv_copy_pages(cache, torch.empty((0, 2), dtype=torch.int32, device="cuda"))
