"""Calls at the edges of what the paged decodes take: shares without a single key, values
that are not finite, thresholds and temperatures at the ends of their range, index lists."""
import math
import random

import pytest
import torch

from long_context_decoding_eta_b200 import _lib as L
from long_context_decoding_eta_b200 import synth
from long_context_decoding_eta_b200.api import EtaDecoder
from long_context_decoding_eta_b200.paged import PagedEtaDecoder, PagedKVCache

from test_gpu_paged_decode import P_EPS, check, make_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["paged", "contiguous"])
def test_values_of_other_rows_stay_out(form):
    """A row's infinite values reach its own output alone: the rows of one block are
    half-full tiles, whose other half held the values of the long rows between them."""
    B, Hkv, d, blk, nb = 64, 4, 64, 64, 16
    gen = torch.Generator().manual_seed(13)
    K, V = (torch.randn(B, Hkv, nb * blk, d, generator=gen).to(torch.bfloat16).cuda()
            for _ in "kv")
    lengths = torch.tensor([blk, nb * blk] * (B // 2), dtype=torch.int32, device="cuda")
    q = torch.randn(B, Hkv, d, generator=gen).to(torch.bfloat16).cuda()

    def paged(x):
        return x.view(B, Hkv, nb, blk, d).transpose(1, 2).reshape(B * nb, Hkv, blk, d)

    if form == "paged":
        c = PagedKVCache(B, Hkv, d, blk, nb, B * nb)
        c.table.copy_(torch.arange(B * nb, dtype=torch.int32).view(B, nb))
        c.lengths.copy_(lengths)
        c.K.copy_(paged(K))
        dec = PagedEtaDecoder(c, Hkv, T=None)
    else:
        dec = EtaDecoder(K, V, lengths, Hkv, blk)

    def run():
        if form == "paged":
            c.V.copy_(paged(V))
        o, _ = dec.dense_decode(q)
        dec.check_status()
        return o.clone()

    want = run()
    V[1::2] = math.inf
    got = run()
    assert torch.equal(got[::2], want[::2])
    assert not torch.isfinite(got[1::2]).any()


def take_status(dec):
    torch.cuda.synchronize()
    s = int(dec.dev_status)
    dec.dev_status.zero_()
    return s


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B", [3, 130])
def test_a_share_without_a_key_is_an_empty_part(B, out):
    """Row 0 keeps its first and last block, row 1 nothing: with at most 4 blocks a share
    some shares hold skipped blocks alone.  6 and 260 (row, KV head) pairs: the shares laid
    out by the decode and by a launch before it."""
    lens = [640, 40, 300] + [70] * (B - 3)
    c = make_cache(lens, 2, 64, 64, seed=7)
    q = torch.randn(B, 4, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    dec = PagedEtaDecoder(c, 4, T=None, out_dtype=out)
    dec.dense_decode(q)
    dec.check_status()
    c.table[0, 1:9] = torch.tensor([-1, c.n_pages] * 4, dtype=torch.int32)
    c.table[1, 0] = c.n_pages + 1
    dec.ws_decode.fill_(0x3F)                # a part that is not written weighs in
    o, lse = dec.dense_decode(q)
    assert take_status(dec) == L.DEVSTAT_BAD_BLOCK
    c.table[0, 1:9] = c.table[1, 0] = 0      # for the oracle's gather: left out below
    blocks = [[[0, 9]] * 2, [[]] * 2, [list(range(5))] * 2] + [[[0, 1]] * 2] * (B - 3)
    assert check(c, q, o, lse, None, None, blocks, p_eps=P_EPS[out]) == 4 * (B - 1)


def test_block_lists_of_a_row_that_was_freed():
    """The lists of the step before: the freed row reads as empty, the others as they are."""
    c = make_cache([640, 500, 300], 2, 64, 64, seed=11)
    dec = PagedEtaDecoder(c, 4, T=None)
    for b, n in enumerate((10, 8, 5)):
        dec.union_idx[b, :, :n] = torch.arange(n, dtype=torch.int32, device="cuda")
        dec.union_cnt[b] = n
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    dec.decode(q)
    dec.check_status()
    c.free([1])
    dec.ws_decode.fill_(0x3F)
    o, lse = dec.decode(q)
    assert take_status(dec) == L.DEVSTAT_BAD_BLOCK
    blocks = [[list(range(n))] * 2 for n in (10, 0, 5)]
    assert check(c, q, o, lse, None, None, blocks, p_eps=2.0 ** -24) == 8


@pytest.mark.parametrize("B", [3, 42])
@pytest.mark.parametrize("engine", ["tcgen05", "fma"])
def test_contiguous_lists_past_a_rows_end(engine, B):
    """The contiguous decode on a list that reaches past a shortened row, and past an empty
    one: the same as with the lists cut at the rows' ends."""
    w = synth.MID.with_(B=B, ctx=1024, seed=51)
    g = {k: (v.cuda() if isinstance(v, torch.Tensor) else v)
         for k, v in synth.generate(w, "cpu").items()}
    dec = EtaDecoder(g["K"], g["V"], g["lengths"], w.Hq, w.blk, T=0.0)
    NB = dec.NB
    dec.tau.fill_(-math.inf)
    dec.union_idx[:] = torch.arange(NB, dtype=torch.int32, device="cuda")
    dec.union_cnt.fill_(NB)
    dec.lengths.copy_(torch.tensor([1024, 0, 256] * (B // 3), dtype=torch.int32))
    L.eta_set_decode_engine(engine)
    try:
        dec.ws_decode.fill_(0x3F)
        dec.decode(g["q"])
        assert take_status(dec) == L.DEVSTAT_BAD_BLOCK
        o, lse = dec.o.clone(), dec.lse.clone()
        dec.union_cnt.copy_(torch.tensor([[NB], [0], [256 // w.blk]] * (B // 3)).expand(B, w.Hkv))
        dec.decode(g["q"])
        dec.check_status()
    finally:
        L.eta_set_decode_engine("auto")
    assert torch.all(o[1::3] == 0) and torch.all(lse[1::3] == -math.inf)
    # cut into other shares: half steps of up to 16 merged parts in numerator and
    # denominator, weights that add up to one, |v| below 7
    assert torch.all((o - dec.o).abs() <= 2 * 16 * 2.0 ** -24 * 7)
    keep = torch.isfinite(lse)
    assert torch.all((lse - dec.lse).abs()[keep] <= 2 * 16 * 2.0 ** -24 * 8)
    assert torch.equal(keep, torch.isfinite(dec.lse))


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [None, 0.05])
@pytest.mark.parametrize("form", ["paged", "shared"])
def test_nan_is_not_an_empty_row(form, T, out):
    """A NaN key or query, or a score of +inf (inf - inf in its softmax), gives NaN outputs
    in the heads that attend to it; the others and empty rows are as without it."""
    Hq, Hkv, d = 4, 2, 64
    lens = [300, 260, 0, 500, 130]
    c = make_cache(lens, Hkv, d, 64, seed=21)
    c.table[1, :3] = c.table[0, :3]
    q = torch.randn(5, Hq, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    q[4, 2, 0] = 1.0
    tau = torch.full((5, Hq), 0.3, device="cuda")
    dec = PagedEtaDecoder(c, Hq, T=T, out_dtype=out)

    def run():
        if form == "paged":
            o, lse = dec.decode(q, tau=tau, all_blocks=True)
        else:
            o, lse = dec.shared_decode(q, [0, 2, 5], [3 * 64, 0], tau=tau)
        dec.check_status()
        return o.clone(), lse.clone()

    o0, l0 = run()
    bad = torch.zeros(5, Hq, dtype=torch.bool, device="cuda")
    c.K[c.table[0, 3].long(), 0, 5] = math.nan      # a key of row 0's own, KV head 0
    bad[0, :2] = True
    q[3, 1, 7] = math.nan                           # a query
    bad[3, 1] = True
    c.K[c.table[4, 2].long(), 1, 1] = 0.0           # row 4, KV head 1: s = +inf in head 2,
    c.K[c.table[4, 2].long(), 1, 1, 0] = math.inf   # whose q[0] is 1; head 3's is set below
    q[4, 3, 0] = -1.0                               # s = -inf: weight 0
    bad[4, 2] = True
    bad[4, 3] = T is not None                       # -inf times the gate's 0
    o, lse = run()
    assert torch.equal(torch.isnan(o).all(-1), bad) and torch.equal(torch.isnan(o).any(-1), bad)
    assert torch.equal(torch.isnan(lse), bad)
    same = ~bad
    same[4, 3] = False                              # its query changed
    assert torch.equal(o[same], o0[same]) and torch.equal(lse[same], l0[same])
    assert torch.all(o[2] == 0) and torch.all(lse[2] == -math.inf)


@pytest.mark.parametrize("engine", ["tcgen05", "fma"])
def test_nan_in_the_contiguous_engines(engine):
    """As above behind contiguous rows; row 1's scores are all NaN."""
    w = synth.MID.with_(B=3, ctx=1024, seed=52)
    g = {k: (v.cuda() if isinstance(v, torch.Tensor) else v)
         for k, v in synth.generate(w, "cpu").items()}
    g["lengths"][2] = 0
    dec = EtaDecoder(g["K"], g["V"], g["lengths"], w.Hq, w.blk, T=0.0)
    L.eta_set_decode_engine(engine)
    try:
        dec.dense_decode(g["q"])
        dec.check_status()
        o, lse = dec.o.clone(), dec.lse.clone()
        g["K"][0, 1, 700] = math.nan
        g["K"][1, 3] = math.nan
        dec.dense_decode(g["q"])
        dec.check_status()
    finally:
        L.eta_set_decode_engine("auto")
    bad = torch.zeros(3, w.Hq, dtype=torch.bool, device="cuda")
    bad[0, w.G:2 * w.G] = bad[1, 3 * w.G:] = True
    assert torch.equal(torch.isnan(dec.lse), bad) and torch.equal(torch.isnan(dec.o).all(-1), bad)
    assert torch.equal(dec.o[~bad], o[~bad]) and torch.equal(dec.lse[~bad], lse[~bad])
    assert torch.all(o[2] == 0) and torch.all(lse[2] == -math.inf)


def test_merge_keeps_nan():
    """A part that is NaN makes the merged row NaN; parts without a key do not count."""
    o = torch.randn(3, 4, 64, device="cuda")
    lse = torch.randn(3, 4, device="cuda")
    lse[1, 0] = lse[0, 1] = -math.inf
    lse[:, 2] = -math.inf
    o[1, 3] = lse[1, 3] = math.nan
    out, l = torch.empty(4, 64, device="cuda"), torch.empty(4, device="cuda")
    L.eta_lse_merge(o, lse, out, l)
    torch.cuda.synchronize()
    assert torch.isnan(out[3]).all() and torch.isnan(l[3])
    assert torch.isfinite(out[:2]).all() and torch.isfinite(l[:2]).all()
    assert torch.all(out[2] == 0) and l[2] == -math.inf


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", ["paged", "shared"])
def test_soft_gate_of_large_scores(form, out):
    """Every key of a row is the same, so that lse = gated score + log n with nothing to
    average the gate's error: scores of about 20, thresholds within 3 T of them."""
    B, Hq, d, n = 48, 8, 64, 64 * 3 + 17
    c = make_cache([n] * B, 1, d, 64, seed=3)
    c.K.zero_()
    c.K[..., 0] = 8.0                        # scale 1/8: the score is q[0]
    c.table[:, :3] = c.table[0, :3]          # one shared prefix
    q = torch.zeros(B, Hq, d)
    q[..., 0] = torch.linspace(16.0, 23.0, Hq)
    q = q.to(torch.bfloat16).cuda()
    T = 8.0
    tau = (q[..., 0].float() + torch.linspace(-24.0, 24.0, B, device="cuda")[:, None]).contiguous()
    dec = PagedEtaDecoder(c, Hq, T=T, out_dtype=out)
    if form == "paged":
        o, lse = dec.decode(q, tau=tau, all_blocks=True)
    else:
        o, lse = dec.shared_decode(q, [0, B], [3 * 64], tau=tau)
    dec.check_status()
    p_eps = P_EPS[out] if form == "paged" else {torch.bfloat16: 2.0 ** -8}.get(out, 2.0 ** -24)
    assert check(c, q, o, lse, tau, T, p_eps=p_eps, gate_eps=2.0 ** -20) == B * Hq


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [None, 0.0, 0.05, 2.0])
def test_lse_is_the_same_for_both_output_types(T, d):
    lens = [64 * 9 + 5, 64 * 9 + 64, 64 * 10 + 1, 90]
    c = make_cache(lens, 2, d, 64, seed=17, poison=True)
    c.table[1:3, :9] = c.table[0, :9]
    gen = torch.Generator().manual_seed(6)
    q = (4 * torch.randn(4, 8, d, generator=gen)).to(torch.bfloat16).cuda()
    tau = (4 * torch.randn(4, 8, generator=gen)).cuda()
    lse = []
    for out in (torch.float32, torch.bfloat16):
        dec = PagedEtaDecoder(c, 8, T=T, out_dtype=out)
        dec.shared_decode(q, [0, 3, 4], [9 * 64, 0], tau=tau)
        dec.check_status()
        lse.append(dec.lse)
    assert torch.isfinite(lse[0]).all() and torch.equal(*lse)


def test_a_threshold_that_is_nan():
    """A soft gate of a NaN threshold is NaN; other heads are as they were."""
    c = make_cache([64 * 3 + 5] * 2, 1, 64, 64, seed=18)
    c.table[1, :3] = c.table[0, :3]
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    tau = torch.full((2, 4), 0.3, device="cuda")
    dec = PagedEtaDecoder(c, 4, T=0.05)
    o = dec.shared_decode(q, [0, 2], [3 * 64], tau=tau)[0].clone()
    tau[1, 2] = math.nan
    bad = torch.isnan(tau)
    for call in (lambda: dec.decode(q, tau=tau, all_blocks=True),
                 lambda: dec.shared_decode(q, [0, 2], [3 * 64], tau=tau)):
        got, lse = call()
        assert torch.isnan(got[bad]).all() and torch.equal(torch.isnan(lse), bad)
        assert torch.isfinite(got[~bad]).all()
    assert torch.equal(dec.o[~bad], o[~bad])


@pytest.mark.parametrize("T", [1e-3, 1e-37, 1e-40])
@pytest.mark.parametrize("form", ["paged", "shared"])
def test_temperatures_near_zero(form, T):
    """A vanishing temperature is the hard gate, and half the score where it meets tau
    (zero keys and zero thresholds: 0)."""
    c = make_cache([64 * 4 + 20, 64 * 4 + 33, 90], 1, 64, 64, seed=4)
    c.table[1, :4] = c.table[0, :4]
    c.K[c.table[2, 0].long()] = 0.0
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    tau = torch.tensor([[0.5, 30.0, -30.0, 1.0], [0.2, 3e4, -3e4, 0.1], [0.0] * 4], device="cuda")
    for out in (torch.float32, torch.bfloat16):
        res = []
        for t in (T, 0.0):
            dec = PagedEtaDecoder(c, 4, T=t, out_dtype=out)
            if form == "paged":
                o, lse = dec.decode(q, tau=tau, all_blocks=True)
            else:
                o, lse = dec.shared_decode(q, [0, 2, 3], [4 * 64, 0], tau=tau)
            dec.check_status()
            res.append((o, lse))
        (o, lse), (ho, hl) = res
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()
        if T < 1e-30:                        # no score is that near its threshold
            n = check(c, q, ho, hl, tau, 0.0, p_eps=2.0 ** -8)
            assert n >= 8
            assert torch.allclose(o.float(), ho.float(), rtol=2.0 ** -7, atol=1e-5)
            assert torch.allclose(lse, hl, atol=1e-5)


def test_types_of_index_tensors():
    """A mask or a float names no rows; numbers past 32 bits are out of range, not wrapped."""
    c = PagedKVCache(4, 1, 64, 64, 4, 12)
    k = torch.randn(40, 1, 64).to(torch.bfloat16).cuda()
    c.append(k, k, [0, 10, 20, 30, 40])
    for bad in ([True, False, True, False], [1.0], [0.5], torch.tensor([True, False, True, False]),
                torch.tensor([1.0]), torch.tensor([True] * 4, device="cuda"),
                torch.zeros(2, device="cuda"), [1 << 31], [-(1 << 31) - 1]):
        with pytest.raises(ValueError):
            c.free(bad)
    assert c.lengths.tolist() == [10] * 4
    c.check_status()
    for x in (torch.tensor([1 << 32]), torch.tensor([1 << 32], device="cuda"),
              torch.tensor([-(1 << 32) + 1], device="cuda")):
        c.free(x)
        torch.cuda.synchronize()
        assert int(c.dev_status) == L.DEVSTAT_BAD_ROW
        c.dev_status.zero_()
    assert c.lengths.tolist() == [10] * 4
    for x in (torch.tensor([0]), torch.tensor([1], dtype=torch.int16, device="cuda"), (2,),
              range(3, 4)):
        c.free(x)
    assert c.lengths.tolist() == [0] * 4


def test_lists_do_not_wait_for_the_stream():
    """Index lists reach the device behind the work that is on the stream already: the calls
    return while it still runs."""
    c = PagedKVCache(4, 1, 64, 64, 4, 12)
    k = torch.randn(300, 1, 64).to(torch.bfloat16).cuda()
    dec = PagedEtaDecoder(c, 2, T=None)
    q = torch.randn(4, 2, 64).to(torch.bfloat16).cuda()

    def calls():
        c.append(k, k, [0, 200, 200, 200, 300])
        c.fork([0, 0], [1, 2])
        dec.shared_decode(q, [0, 3, 4], [192, 0])
        c.copy_pages(torch.tensor([0]), torch.tensor([11]))
        c.free(range(4))

    calls()                                   # allocates, loads the kernels
    torch.cuda.synchronize()
    c.check_status()
    done = torch.cuda.Event()
    torch.cuda._sleep(2_000_000_000)          # about a second
    calls()
    done.record()
    assert not done.query()
    done.synchronize()
    c.check_status()
    dec.check_status()
    assert int(c.n_free) == 12 and c.lengths.tolist() == [0] * 4


def test_lists_are_refused_in_a_capture():
    c = PagedKVCache(4, 1, 64, 64, 4, 12)
    dec = PagedEtaDecoder(c, 2, T=None)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0], dtype=torch.int32, device="cuda")
    host = rows.cpu()
    c.free(rows)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.free(rows)
        for call in (lambda: c.free([0]), lambda: c.fork([0], rows), lambda: c.free(host),
                     lambda: dec.shared_decode(q, [0, 4], [0])):
            with pytest.raises(ValueError, match="captur"):
                call()
    g.replay()
    torch.cuda.synchronize()
    c.check_status()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_hard_gated_lists_against_64_bits(out):
    """How many heads are compared counts here: a head of n keys in its blocks is left out
    for a near-tie with probability 0.4 n 4 ds at most (scores of density 0.4, ds = 132 *
    2^-24 * 10), 0.12 for the longest list and 0.04 on average; four in five is far below."""
    lens = [1500, 130, 64, 0, 900, 333]
    Hq, Hkv, d, blk = 16, 4, 128, 64
    c = make_cache(lens, Hkv, d, blk, seed=23, poison=True)
    rng = random.Random(5)
    dec = PagedEtaDecoder(c, Hq, T=0.0, out_dtype=out)
    blocks = []
    for b, n in enumerate(lens):
        nb = -(-n // blk)
        row = [sorted(rng.sample(range(nb), rng.randint(min(1, nb), nb))) for _ in range(Hkv)]
        for g in range(Hkv):
            dec.union_idx[b, g, :len(row[g])] = torch.tensor(row[g], dtype=torch.int32).cuda()
            dec.union_cnt[b, g] = len(row[g])
        blocks.append(row)
    gen = torch.Generator().manual_seed(24)
    q = torch.randn(len(lens), Hq, d, generator=gen).to(torch.bfloat16).cuda()
    tau = (0.3 + 0.5 * torch.randn(len(lens), Hq, generator=gen)).cuda()
    o, lse = dec.decode(q, tau=tau)
    dec.check_status()
    assert check(c, q, o, lse, tau, 0.0, blocks, p_eps=P_EPS[out]) >= 0.8 * 5 * Hq


def test_hard_gate_after_fork_free_and_compact():
    """Both decodes of rows that were appended, forked, freed, compacted and forked again;
    near-ties as above, 420 keys a row: 0.03 a head."""
    B, Hq, Hkv, d, blk = 6, 8, 2, 128, 64
    c = PagedKVCache(B, Hkv, d, blk, 12, 40)
    gen = torch.Generator().manual_seed(25)

    def tokens(n):
        return [torch.randn(n, Hkv, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]

    n0 = 5 * blk + 17
    c.append(*tokens(n0 + 100), [0, n0, n0, n0, n0, n0 + 100, n0 + 100])
    c.fork([0, 0, 0], [1, 2, 3])
    c.append(*tokens(200), [0, 40, 80, 120, 160, 200, 200])
    c.free([0, 4])
    c.compact()
    c.fork([2], [0])
    c.append(*tokens(4), [0, 1, 2, 3, 4, 4, 4])
    q = torch.randn(B, Hq, d, generator=gen).to(torch.bfloat16).cuda()
    tau = (0.3 + 0.5 * torch.randn(B, Hq, generator=gen)).cuda()
    dec = PagedEtaDecoder(c, Hq, T=0.0)
    assert c.lengths.tolist() == [n0 + 41] * 4 + [0, 0]
    for call in (lambda: dec.shared_decode(q, [0, 4, 6], [n0, 0], tau=tau),
                 lambda: dec.decode(q, tau=tau, all_blocks=True)):
        o, lse = call()
        c.check_status()
        dec.check_status()
        assert check(c, q, o, lse, tau, 0.0, p_eps=2.0 ** -24) >= 0.8 * 4 * Hq
