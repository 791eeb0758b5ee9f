"""Page operations of the paged cache on the GPU against the plain model of the rules:
every word of the bookkeeping after every call, and every byte of the pools."""
import random

import numpy as np
import pytest
import torch

from long_context_decoding_eta_b200 import _lib as L
from long_context_decoding_eta_b200.paged import PagedKVCache

from paged_testlib import PageModel

pytestmark = pytest.mark.gpu


class Both:
    """A cache and its model, and the pools' expected contents on the host."""

    def __init__(self, B, Hkv, d, blk, max_pages, n_pages, seed=0):
        self.c = PagedKVCache(B, Hkv, d, blk, max_pages, n_pages)
        self.m = PageModel(B, blk, max_pages, n_pages)
        self.g = torch.Generator().manual_seed(seed)
        for t in (self.c.K, self.c.V):
            t.copy_(torch.randn(t.shape, generator=self.g).to(torch.bfloat16))
        self.K, self.V = self.c.K.cpu(), self.c.V.cpu()
        self.Hkv, self.d = Hkv, d

    def append(self, counts, cu=None, n_new=None):
        cu = list(np.concatenate([[0], np.cumsum(counts)])) if cu is None else cu
        n_new = int(cu[-1]) if n_new is None else n_new
        k = torch.randn(n_new, self.Hkv, self.d, generator=self.g).to(torch.bfloat16)
        v = torch.randn(n_new, self.Hkv, self.d, generator=self.g).to(torch.bfloat16)
        self.m.tokens = {}
        self.m.append([int(x) for x in cu], n_new)
        self.c.append(k.cuda(), v.cuda(), cu)
        for (page, slot), t in self.m.tokens.items():
            self.K[page, :, slot] = k[t]
            self.V[page, :, slot] = v[t]

    def _move(self):
        K0, V0 = self.K.clone(), self.V.clone()
        for f, t, n in self.m.moves:
            self.K[t, :, :n] = K0[f, :, :n]
            self.V[t, :, :n] = V0[f, :, :n]

    def fork(self, src, dst):
        self.m.fork(src, dst)
        self._move()
        self.c.fork(src, dst)

    def free(self, rows):
        self.m.free(rows)
        self.c.free(rows)

    def compact(self):
        self.m.compact()
        self._move()
        self.c.compact()

    def check(self, status=0):
        torch.cuda.synchronize()
        assert int(self.c.dev_status) == self.m.status == status
        self.m.check(self.c)
        assert torch.equal(self.c.K.cpu(), self.K)
        assert torch.equal(self.c.V.cpu(), self.V)


@pytest.mark.parametrize("B,Hkv,d,blk", [(1, 1, 64, 64), (5, 2, 128, 64), (3, 4, 64, 128),
                                         (70, 1, 128, 128), (1030, 1, 64, 64)])
def test_append_fork_free_compact_in_random_order(B, Hkv, d, blk):
    t = Both(B, Hkv, d, blk, 5, 4 * B + 3, seed=B)
    rng = random.Random(B)
    t.check()
    for _ in range(12):
        free_rows = [b for b in range(B) if t.m.len[b] == 0]
        counts = [min(rng.choice((0, 1, 1, 2, blk - 1, blk, blk + 1)),
                      5 * blk - t.m.len[b]) for b in range(B)]
        t.append(counts)
        if free_rows and B > 1:
            dst = [b for b in free_rows if t.m.len[b] == 0]
            if dst:
                t.fork([rng.randrange(B) for _ in dst], dst)
        t.free(rng.sample(range(B), rng.randint(1, B)))
        if rng.random() < 0.4:
            t.compact()
    torch.cuda.synchronize()
    # the pool may have run out on the way: rows were then refused by both alike
    t.check(t.m.status)
    assert t.m.status in (0, L.DEVSTAT_NO_PAGE)
    t.free(list(range(B)))
    t.compact()
    t.check(t.m.status)
    assert int(t.c.n_free) == 4 * B + 3


@pytest.mark.parametrize("n", [1, 63, 64, 65, 64 * 9])
def test_append_sizes_at_page_borders(n):
    t = Both(3, 2, 128, 64, 10, 40)
    t.append([n, 0, 1])
    t.check()
    t.append([0, n, 1])
    t.append([1, 1, 1])
    t.check()


def test_append_one_token_a_row_without_offsets():
    t = Both(4, 2, 64, 64, 2, 8)
    k = torch.randn(4, 2, 64).to(torch.bfloat16)
    t.m.append([0, 1, 2, 3, 4], 4)
    t.c.append(k.cuda(), k.cuda())
    for b in range(4):
        t.K[t.m.pages[b][0], :, 0] = k[b]
        t.V[t.m.pages[b][0], :, 0] = k[b]
    t.check()


def test_append_refuses_rows_past_their_capacity_and_bad_offsets():
    t = Both(4, 1, 64, 64, 2, 20)
    t.append([128, 100, 0, 0])
    t.append([1, 28, 129, 128])              # rows 0 and 2 do not fit
    t.check(L.DEVSTAT_BAD_LENGTH)
    t.m.status = 0
    t.c.dev_status.zero_()
    t.free([0, 1, 2, 3])


@pytest.mark.parametrize("cu", [[0, 5, 3, 9, 10], [0, 1, 2, 3, 11], [-1, 1, 2, 3, 10],
                                [0, 10, 10, 10, 9]])
def test_append_with_offsets_out_of_order_changes_nothing(cu):
    t = Both(4, 1, 64, 64, 2, 20)
    t.append([3, 70, 0, 0])
    t.append(None, cu=cu, n_new=10)
    t.check(L.DEVSTAT_BAD_LENGTH)
    assert t.m.len == [3, 70, 0, 0]


def test_append_serves_rows_in_order_while_pages_last():
    t = Both(5, 1, 64, 64, 4, 5)
    t.append([64, 10, 0, 0, 0])
    t.append([100, 50, 130, 1, 0])           # 2 + 0 + 3 + 1 pages, 3 are left
    t.check(L.DEVSTAT_NO_PAGE)
    assert t.m.len == [164, 60, 0, 0, 0]     # row 3's page comes behind row 2's request
    with pytest.raises(L.EtaError) as e:
        t.c.check_status()
    assert e.value.code == 8
    t.m.status = 0
    t.append([0, 4, 0, 64, 0])
    t.check()


def test_append_to_a_shared_partial_page_is_refused():
    t = Both(2, 1, 64, 64, 2, 8)
    t.append([10, 0])
    t.c.ref[t.m.pages[0][0]] = 2
    t.m.ref[t.m.pages[0][0]] = 2
    t.append([1, 1])
    t.check(L.DEVSTAT_BAD_ROW)
    assert t.m.len == [10, 1]


def test_fork_refusals():
    t = Both(6, 2, 64, 64, 3, 30)
    t.append([100, 64, 0, 0, 0, 0])
    # a dst named twice, one that is not empty, numbers out of range, itself
    t.fork([0, 1, 0, 0, -1, 0], [2, 2, 1, 6, 3, 0])
    t.check(L.DEVSTAT_BAD_ROW)
    assert t.m.len == [100, 64, 100, 0, 0, 0]
    # a pair's source that is another pair's dst counts as it was: empty
    t.fork([0, 3], [3, 4])
    t.check(L.DEVSTAT_BAD_ROW)
    assert t.m.len == [100, 64, 100, 100, 0, 0]


def test_fork_when_pages_run_out():
    t = Both(5, 1, 128, 128, 2, 4)
    t.append([130, 128, 0, 0, 0])            # 3 pages
    t.fork([0, 0, 1], [2, 3, 4])             # one page left for the first pair's tail
    t.check(L.DEVSTAT_NO_PAGE)
    assert t.m.len == [130, 128, 130, 0, 128]


def test_free_twice_out_of_range_and_empty():
    t = Both(4, 1, 64, 64, 3, 12)
    t.append([150, 64, 1, 0])
    t.fork([0], [3])
    t.free([0, 0, 3, 1, 0][:4])
    t.check()
    t.free([-1, 4, 0, 2])
    t.check(L.DEVSTAT_BAD_ROW)
    assert int(t.c.n_free) == 12


def test_append_to_a_fork_leaves_its_source_alone():
    t = Both(3, 2, 128, 64, 4, 16)
    t.append([100, 0, 0])
    t.fork([0, 0], [1, 2])
    t.append([3, 30, 64])
    t.check()
    assert t.m.ref[t.m.pages[0][0]] == 3     # the whole page is shared by all three
    t.free([0])
    t.append([0, 1, 1])
    t.check()


def test_compact_moves_shared_pages_once():
    t = Both(6, 2, 64, 64, 4, 64)
    t.append([200, 130, 64, 0, 0, 0])
    t.fork([1, 1, 0], [3, 4, 5])
    t.free([0, 2])
    t.compact()
    t.check()
    n_live = 64 - int(t.c.n_free)
    assert int(t.c.table.max()) == n_live - 1
    t.compact()                              # nothing is left to move
    assert t.m.moves == []
    t.check()


def test_compact_of_empty_and_full_pools():
    t = Both(2, 1, 64, 64, 4, 8)
    t.compact()
    t.check()
    t.append([256, 256])
    t.compact()
    t.check()


def test_compact_with_an_inconsistent_header_changes_nothing():
    t = Both(2, 1, 64, 64, 4, 8)
    t.append([100, 100])
    t.free([0])
    before = t.c.state.clone()
    t.c.state[0] += 1
    t.c.compact()
    torch.cuda.synchronize()
    assert int(t.c.dev_status) == L.DEVSTAT_BAD_BLOCK
    before[0] += 1
    assert torch.equal(t.c.state, before)
    assert torch.equal(t.c.K.cpu(), t.K)


@pytest.mark.parametrize("n_pages", [2 * 4096 + 77, 8 * 4096 + 130])
def test_many_chunks_of_pages(n_pages):
    """More pages than one CTA of the compaction's scan takes, ends inside a chunk."""
    B = 64
    t = Both(B, 1, 64, 64, 160, n_pages, seed=5)
    rng = random.Random(3)
    t.append([rng.randint(1, 125 * 64) for _ in range(B)])
    t.free([b for b in range(B) if b % 3 != 1])
    t.compact()
    t.check()


@pytest.mark.parametrize("d,Hkv,blk", [(64, 1, 64), (128, 3, 128)])
def test_copy_pages(d, Hkv, blk):
    c = PagedKVCache(1, Hkv, d, blk, 1, 40)
    for x in (c.K, c.V):
        x.copy_(torch.randn(x.shape).to(torch.bfloat16))
    K, V = c.K.clone(), c.V.clone()
    state = c.state.clone()
    src, dst = [0, 0, 39, 7], [1, 2, 30, 8]
    c.copy_pages(src, dst)
    K[dst], V[dst] = K[src], V[src]
    torch.cuda.synchronize()
    c.check_status()
    assert torch.equal(c.K, K) and torch.equal(c.V, V) and torch.equal(c.state, state)
    # a dst named twice (the first pair counts), a dst that is a src, out of range
    c.copy_pages([3, 4, 5, 6, -1, 40, 9], [10, 10, 4, 40, 11, 12, 9])
    K[10], V[10] = K[3], V[3]
    torch.cuda.synchronize()
    assert int(c.dev_status) == L.DEVSTAT_BAD_ROW
    assert torch.equal(c.K, K) and torch.equal(c.V, V)


def test_many_copies():
    """More pairs than a CTA compares by itself."""
    n_pages, n = 5000, 2200
    c = PagedKVCache(1, 1, 64, 64, 1, n_pages)
    gen = torch.Generator().manual_seed(6)
    for x in (c.K, c.V):
        x.copy_(torch.randn(x.shape, generator=gen).to(torch.bfloat16))
    K, V = c.K.clone(), c.V.clone()
    perm = torch.randperm(n_pages, generator=gen)
    src, dst = perm[:n].clone(), perm[n:2 * n].clone()
    c.copy_pages(src, dst)
    K[dst.cuda()], V[dst.cuda()] = K[src.cuda()], V[src.cuda()]
    torch.cuda.synchronize()
    c.check_status()
    assert torch.equal(c.K, K) and torch.equal(c.V, V)
    dst[n - 1], dst[5], dst[7] = dst[0], src[3], -1      # refused, all three
    c.K.copy_(V)
    K = V.clone()
    ok = torch.ones(n, dtype=torch.bool)
    ok[[n - 1, 5, 7]] = False
    c.copy_pages(src, dst)
    K[dst[ok].cuda()] = K[src[ok].cuda()]
    torch.cuda.synchronize()
    assert int(c.dev_status) == L.DEVSTAT_BAD_ROW
    assert torch.equal(c.K, K)


def test_calls_leave_the_workspace_ready():
    """Append, fork and free one after another many times: the count of finished CTAs and
    the page bitmap are left as every call needs them."""
    t = Both(12, 1, 64, 64, 40, 300)
    for i in range(30):
        t.append([(i * 7 + b) % 90 for b in range(6)] + [0] * 6)
        t.fork(list(range(6)), list(range(6, 12)))
        t.free([b for b in range(12) if (b + i) % 2 or b > 5])
    t.check()


def test_snapshot_and_graph_replay():
    """One decode step's append captured once and replayed: pages are taken as the
    lengths grow; a copy of the state takes the cache back."""
    t = Both(3, 1, 64, 64, 4, 12)
    t.append([60, 0, 63])
    snap = t.c.state.clone()
    k = torch.randn(3, 1, 64).to(torch.bfloat16)
    kd = k.cuda()
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        t.c.append(kd, kd, cu)               # warm the launch path, then take it back
        t.c.state.copy_(snap)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            t.c.append(kd, kd, cu)
    torch.cuda.current_stream().wait_stream(s)
    t.c.state.copy_(snap)
    for _ in range(6):
        g.replay()
        t.m.tokens = {}
        t.m.append([0, 1, 2, 3], 3)
        for (page, slot), i in t.m.tokens.items():
            t.K[page, :, slot] = k[i]
            t.V[page, :, slot] = k[i]
    t.check()
    assert t.m.len == [66, 6, 69]
