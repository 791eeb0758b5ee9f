"""Decode of batches whose rows share prefixes: against attention in 64 bits, with the
error bounds of paged_testlib, over each row's own tokens."""
import math
import random

import pytest
import torch

from long_context_decoding_eta_b200 import _lib as L
from long_context_decoding_eta_b200.paged import PagedEtaDecoder, PagedKVCache

from test_gpu_paged_decode import check, make_cache

pytestmark = pytest.mark.gpu

# weights: one bf16 term (half a step, 2^-8 at most) or the sum of three (2^-24)
P_EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
GATE_EPS = {torch.bfloat16: 2.0 ** -10, torch.float32: 2.0 ** -20}


def shared_cache(groups, Hkv, d, blk, seed=0, poison=True):
    """groups: (prefix blocks, [tokens of each row]); a row longer than the prefix holds
    the pages of the group's first such row there.  Returns the cache, group_off, prefix."""
    lens = [n for _, rows in groups for n in rows]
    c = make_cache(lens, Hkv, d, blk, seed=seed, poison=poison)
    off, pre, b = [0], [], 0
    for nb, rows in groups:
        long_rows = [b + i for i, n in enumerate(rows) if n >= nb * blk]
        for r in long_rows[1:]:
            c.table[r, :nb] = c.table[long_rows[0], :nb]
        b += len(rows)
        off.append(b)
        pre.append(nb * blk)
    return c, off, pre


def run_and_check(c, Hq, off, pre, T, out, seed=1, sharp=1.0, lowest=0.9):
    B = c.B
    gen = torch.Generator().manual_seed(seed)
    q = (sharp * torch.randn(B, Hq, c.d, generator=gen)).to(torch.bfloat16).cuda()
    tau = (0.3 + 0.5 * torch.randn(B, Hq, generator=gen)).cuda()
    dec = PagedEtaDecoder(c, Hq, T=T, out_dtype=out)
    o, lse = dec.shared_decode(q, off, pre, tau=tau)
    dec.check_status()
    seen = check(c, q, o, lse, None if T is None else tau, T, p_eps=P_EPS[out],
                 gate_eps=GATE_EPS[out])
    assert seen >= lowest * Hq * sum(n > 0 for n in c.lengths.tolist())
    return dec, q, tau


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [None, 0.0, 0.05])
@pytest.mark.parametrize("Hq,Hkv,d,blk", [(4, 1, 64, 64), (8, 8, 128, 128), (16, 2, 128, 64),
                                          (4, 2, 64, 128)])
def test_groups_of_every_kind(Hq, Hkv, d, blk, T, out):
    groups = [
        (7, [7 * blk + 1, 7 * blk + 130, 7 * blk, 8 * blk]),       # odd number of pages
        (0, [3, 200]),                                            # nothing shared
        (2, [2 * blk + 5]),                                       # a group of one
        (3, [0, 3 * blk - 1, 3 * blk + 64, 3 * blk + 65, 1]),     # rows that do not share
        (1, [blk, blk]),                                          # the prefix is all
        (4, [10, 4 * blk]),                                       # one row long enough
        (0, [0, 0]),
    ]
    c, off, pre = shared_cache(groups, Hkv, d, blk, seed=Hq + d)
    run_and_check(c, Hq, off, pre, T, out)


@pytest.mark.parametrize("Hq,Hkv,d,rows", [(8, 1, 128, 16), (8, 1, 128, 17), (8, 1, 64, 32),
                                           (8, 1, 128, 33), (4, 2, 64, 150), (1, 1, 128, 129),
                                           (2, 2, 64, 300)])
def test_pairs_at_the_borders_of_a_tile(Hq, Hkv, d, rows):
    """rows * G around 128 and 256 (row, head) pairs, and several items a group."""
    rng = random.Random(rows)
    groups = [(5, [5 * 64 + rng.choice((0, 1, 64, 100)) for _ in range(rows)]), (2, [129, 140])]
    c, off, pre = shared_cache(groups, Hkv, d, 64, seed=rows)
    run_and_check(c, Hq, off, pre, None, torch.float32)
    run_and_check(c, Hq, off, pre, 0.0, torch.bfloat16)


@pytest.mark.parametrize("sharp", [0.0, 0.01, 12.0])
def test_sharp_and_flat_scores(sharp):
    """Equal scores, and scores whose running maximum grows by far more than the bound
    below which accumulators are left as they are."""
    c, off, pre = shared_cache([(40, [40 * 64 + 33] * 5), (0, [3000])], 2, 128, 64, seed=2)
    run_and_check(c, 8, off, pre, None, torch.float32, sharp=sharp)
    run_and_check(c, 8, off, pre, None, torch.bfloat16, sharp=sharp)


def test_growing_scores_rescale_the_accumulators():
    c, off, pre = shared_cache([(30, [30 * 64 + 70, 30 * 64])], 1, 128, 64, poison=False)
    nb = c.table.shape[1]
    q0 = torch.randn(128).to(torch.bfloat16)
    # keys along the query, longer from page to page: every tile has a new maximum
    for j in range(nb):
        page = int(c.table[0, j])
        c.K[page, 0] = (q0.cuda()[None] * 0.1 * j + 0.1 * c.K[page, 0]).to(torch.bfloat16)
    q = q0.cuda().expand(2, 4, 128).contiguous()
    for out in (torch.float32, torch.bfloat16):
        dec = PagedEtaDecoder(c, 4, T=None, out_dtype=out)
        o, lse = dec.shared_decode(q, off, pre)
        dec.check_status()
        assert check(c, q, o, lse, None, None, p_eps=P_EPS[out]) == 8


def test_thresholds_at_the_ends_of_their_range():
    """tau = -inf and lowest: no gate; +inf and highest: every gated score is 0."""
    c, off, pre = shared_cache([(3, [3 * 64 + 10, 3 * 64 + 99])], 1, 64, 64, seed=5)
    q = torch.randn(2, 4, 64).to(torch.bfloat16).cuda()
    big = torch.finfo(torch.float32).max
    tau = torch.tensor([[-math.inf, -big, math.inf, big]] * 2).cuda()
    for T in (0.0, 0.05):
        for out in (torch.float32, torch.bfloat16):
            dec = PagedEtaDecoder(c, 4, T=T, out_dtype=out)
            o, lse = dec.shared_decode(q, off, pre, tau=tau)
            dec.check_status()
            plain = PagedEtaDecoder(c, 4, T=None, out_dtype=out)
            po, pl = plain.shared_decode(q, off, pre)
            assert torch.allclose(o[:, :2].float(), po[:, :2].float(), rtol=2.0 ** -7, atol=1e-3)
            for b in range(2):
                n = int(c.lengths[b])
                assert torch.allclose(lse[b, 2:].cpu(), torch.tensor(math.log(n)), atol=1e-5)


def test_long_prefix_and_many_rows():
    rng = random.Random(8)
    groups = [(200, [200 * 128 + rng.randint(0, 300) for _ in range(20)]),
              (77, [77 * 128 + rng.randint(0, 300) for _ in range(3)]),
              (0, [15000])]
    c, off, pre = shared_cache(groups, 2, 128, 128, seed=12)
    run_and_check(c, 8, off, pre, 0.05, torch.bfloat16)
    run_and_check(c, 8, off, pre, None, torch.float32)


def test_pages_past_32_bit_offsets():
    """Two rows whose shared and own pages lie past 2^32 bytes of the pools."""
    Hkv, d, blk, n_pages = 4, 128, 128, 40000          # 5.2 GB of keys
    c = PagedKVCache(2, Hkv, d, blk, 20, n_pages)
    ids = torch.arange(n_pages - 40, n_pages, dtype=torch.int32).flip(0).cuda()
    gen = torch.Generator().manual_seed(5)
    k, v = (torch.randn(40, Hkv, blk, d, generator=gen).to(torch.bfloat16).cuda() for _ in "kv")
    c.K[ids.long()], c.V[ids.long()] = k, v
    small = make_cache([20 * blk - 7] * 2, Hkv, d, blk)
    order = small.table.view(-1).long()
    small.K[order], small.V[order] = k, v
    for x, first in ((c, ids), (small, small.table.view(-1).clone())):
        x.table.copy_(first.view(2, 20))
        x.table[1, :15] = x.table[0, :15]
        x.lengths.fill_(20 * blk - 7)
    q = torch.randn(2, 8, d, generator=gen).to(torch.bfloat16).cuda()
    dec = PagedEtaDecoder(c, 8, T=None)
    o, lse = dec.shared_decode(q, [0, 2], [15 * blk])
    dec.check_status()
    assert check(small, q, o, lse, None, None, p_eps=2.0 ** -24) == 16


def test_the_same_bits_on_every_call():
    c, off, pre = shared_cache([(50, [50 * 64 + 7] * 9), (10, [700, 800])], 2, 128, 64, seed=3)
    dec, q, tau = run_and_check(c, 8, off, pre, 0.05, torch.float32)
    o, lse = dec.o.clone(), dec.lse.clone()
    for _ in range(5):
        dec.o.fill_(float("nan"))
        dec.shared_decode(q, off, pre, tau=tau)
        assert torch.equal(dec.o, o) and torch.equal(dec.lse, lse)


def test_prefix_is_rounded_down_to_whole_pages():
    c, off, _ = shared_cache([(2, [200, 300])], 1, 64, 64, seed=4)
    run_and_check(c, 4, off, [2 * 64 + 63], None, torch.float32)


def test_bad_groups_lengths_and_pages():
    c, off, pre = shared_cache([(3, [3 * 64 + 10, 3 * 64 + 20]), (2, [150, 140])], 1, 64, 64)
    q = torch.randn(4, 4, 64).to(torch.bfloat16).cuda()
    dec = PagedEtaDecoder(c, 4, T=None)

    def status():
        torch.cuda.synchronize()
        s = int(dec.dev_status)
        dec.dev_status.zero_()
        return s

    # offsets out of order, out of range, not from 0 to B: rows are read by themselves
    for bad in ([0, 3, 2], [0, 2, 5], [-1, 2, 4], [1, 2, 4], [0, 2, 3]):
        o, lse = dec.shared_decode(q, bad, pre)
        assert status() == L.DEVSTAT_BAD_ROW, bad
        assert check(c, q, o, lse, None, None, p_eps=2.0 ** -24) == 16
    # a prefix out of range is clamped: no row is that long, none shares
    for bad in ([-5, 0], [1 << 30, 0]):
        o, lse = dec.shared_decode(q, off, bad)
        assert status() == L.DEVSTAT_BAD_LENGTH
        assert check(c, q, o, lse, None, None, p_eps=2.0 ** -24) == 16
    # pages out of range, in the prefix and in a row's own part: their keys are left out
    c.table[0, 1] = c.n_pages
    c.table[3, 2] = -7
    o, lse = dec.shared_decode(q, off, pre)
    assert status() == L.DEVSTAT_BAD_BLOCK
    c.table[0, 1] = c.table[3, 2] = 0
    blocks = [[[0, 2, 3]], [[0, 2, 3]], [[0, 1, 2]], [[0, 1]]]
    assert check(c, q, o, lse, None, None, blocks, p_eps=2.0 ** -24) == 16


def test_graph_replay_follows_lengths_and_groups():
    c, off, pre = shared_cache([(4, [4 * 64 + 10, 4 * 64 + 20]), (2, [150, 140])], 1, 64, 64)
    q = torch.randn(4, 4, 64).to(torch.bfloat16).cuda()
    dec = PagedEtaDecoder(c, 4, T=None)
    off_d = torch.tensor(off, dtype=torch.int32).cuda()
    pre_d = torch.tensor(pre, dtype=torch.int32).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dec.shared_decode(q, off_d, pre_d)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            dec.shared_decode(q, off_d, pre_d)
    torch.cuda.current_stream().wait_stream(s)
    for lens, pre2 in (([266, 276, 150, 140], [256, 128]), ([257, 257, 0, 128], [192, 64]),
                       ([1, 300, 128, 128], [0, 128])):
        c.lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        pre_d.copy_(torch.tensor(pre2, dtype=torch.int32))
        c.K.nan_to_num_(0.5, 0.5, 0.5)
        c.V.nan_to_num_(0.5, 0.5, 0.5)
        g.replay()
        dec.check_status()
        check(c, q, dec.o, dec.lse, None, None, p_eps=2.0 ** -24)


def test_two_decoders_on_two_streams():
    cs = [shared_cache([(60, [60 * 64 + 9] * 6), (0, [900])], 2, 128, 64, seed=s) for s in (1, 2)]
    work = []
    for c, off, pre in cs:
        # near-ties are left out: 3,849 keys a row, scores of density 0.4 at most, a
        # width of 4 ds, ds = 132 * 2^-24 * A with A <= 12: a head has none with probability
        # e^(-3849 * 0.4 * 4 ds) >= 0.55, and three sigma of 56 heads are 0.2
        dec, q, tau = run_and_check(c, 8, off, pre, 0.0, torch.float32, seed=7, lowest=0.35)
        work.append((dec, q, tau, dec.o.clone(), off, pre, torch.cuda.Stream()))
        dec.o.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for dec, q, tau, _, off, pre, s in work:
            with torch.cuda.stream(s):
                dec.shared_decode(q, off, pre, tau=tau)
    torch.cuda.synchronize()
    for dec, _, _, want, _, _, _ in work:
        assert torch.equal(dec.o, want)


def test_a_serving_run():
    """A prompt, its continuations, several steps, one dropped and replaced, compaction:
    after every step the shared decode and the plain paged decode agree with 64 bits."""
    B, Hq, Hkv, d, blk = 6, 8, 2, 128, 64
    c = PagedKVCache(B, Hkv, d, blk, 12, 40)
    gen = torch.Generator().manual_seed(0)

    def tokens(n):
        return [torch.randn(n, Hkv, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]

    n0 = 5 * blk + 17
    c.append(*tokens(n0 + 100), [0, n0, n0, n0, n0, n0 + 100, n0 + 100])
    c.fork([0, 0, 0], [1, 2, 3])
    dec = PagedEtaDecoder(c, Hq, T=0.0)
    bias = torch.full((Hq,), 0.4, device="cuda")
    W = torch.zeros(Hq * d, Hq, device="cuda")
    off, pre = [0, 4, 6], [n0, 0]
    for step in range(5):
        c.append(*tokens(5), [0, 1, 2, 3, 4, 5, 5])
        q = torch.randn(B, Hq, d, generator=gen).to(torch.bfloat16).cuda()
        if step == 2:
            c.free([0, 4])
            c.compact()
            c.fork([2], [0])
        dec.build_meta()
        dec.predict_tau(q, W, bias)
        o, lse = dec.shared_decode(q, off, pre)
        c.check_status()
        dec.check_status()
        check(c, q, o, lse, dec.tau, 0.0, p_eps=P_EPS[torch.float32])
        dec.screen(q)
        o, lse = dec.decode(q, all_blocks=True)
        dec.check_status()
        check(c, q, o, lse, dec.tau, 0.0, p_eps=2.0 ** -24)
    assert int(c.n_free) == 40 - int((c.ref > 0).sum())


def test_layer_refuses_wrong_groups():
    c, off, pre = shared_cache([(2, [200, 300])], 1, 64, 64)
    dec = PagedEtaDecoder(c, 4, T=0.0)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    for bad_off, bad_pre in (([0], []), ([0, 1, 2, 2], [0, 0, 0]), ([0, 2], [64, 64])):
        with pytest.raises(ValueError):
            dec.shared_decode(q, bad_off, bad_pre)
    with pytest.raises(ValueError):
        dec.shared_decode(q.float(), off, pre)
    with pytest.raises(ValueError):
        dec.shared_decode(q, off, pre, tau=torch.zeros(2, 4))
    for bad in (dict(W=torch.zeros(4, 64, device="cuda")), dict(), dict(tau_const=torch.zeros(4)),
                dict(W=torch.zeros(256, 4, device="cuda"), bias=torch.zeros(2, device="cuda"))):
        with pytest.raises(ValueError):
            dec.predict_tau(q, **bad)


def test_lists_and_a_given_stream():
    """Index lists become device tensors of the stream that reads them, not of the current
    one, where the next allocation could take their memory while they are in use."""
    c = PagedKVCache(6, 2, 128, 64, 32, 80)
    kv = [torch.randn(1929 + 900, 2, 128).to(torch.bfloat16).cuda() for _ in range(2)]
    c.append(*kv, [0] + [1929] * 5 + [2829])
    c.fork([0] * 4, [1, 2, 3, 4])
    off, pre = [0, 5, 6], [1929, 0]
    dec, q, tau = run_and_check(c, 8, off, pre, None, torch.float32)
    want, lens = dec.o.clone(), c.lengths.tolist()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        c.free([1, 2], stream=s)
        c.fork([0, 0], [1, 2], stream=s)
        dec.shared_decode(q, off, pre, tau=tau, stream=s)
        junk = [torch.full((7,), 1 << 20, dtype=torch.int32, device="cuda") for _ in range(4)]
    s.synchronize()
    c.check_status()
    dec.check_status()
    assert len(junk) == 4 and c.lengths.tolist() == lens
    assert torch.equal(dec.o, want)


def test_a_captured_call_outlives_calls_with_other_groups():
    c, off, pre = shared_cache([(4, [4 * 64 + 10, 4 * 64 + 20]), (2, [150, 140])], 1, 64, 64)
    q = torch.randn(4, 4, 64).to(torch.bfloat16).cuda()
    dec = PagedEtaDecoder(c, 4, T=None)
    with pytest.raises(ValueError, match="before it is captured"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            dec.build_meta()
    off_d = torch.tensor([0, 4], dtype=torch.int32).cuda()
    pre_d = torch.tensor([0], dtype=torch.int32).cuda()
    dec.shared_decode(q, off_d, pre_d)
    want = dec.o.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec.shared_decode(q, off_d, pre_d)
    at = dec.ws_shared.data_ptr()
    dec.shared_decode(q, [0, 1, 2, 3, 4], [0, 0, 0, 0])
    assert dec.ws_shared.data_ptr() == at
    dec.o.zero_()
    g.replay()
    dec.check_status()
    assert torch.equal(dec.o, want)


def test_many_more_rows_than_threads_of_the_plan():
    """1,100 rows and groups: every loop of the work list's kernel takes a second turn."""
    rng = random.Random(3)
    groups = [(1, [64 + rng.randint(0, 80), 64 + rng.randint(0, 80)]) if i % 10 == 0 else
              (0, [rng.randint(0, 130)]) for i in range(1030)]
    c, off, pre = shared_cache(groups, 1, 64, 64, seed=4)
    assert c.B > 1024 and len(pre) > 1024
    run_and_check(c, 2, off, pre, None, torch.float32)
