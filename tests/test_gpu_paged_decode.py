"""Decode over a paged cache: against attention in 64 bits with error bounds derived in
paged_testlib, and against the contiguous cache's calls (the same bits where the work is
split alike)."""
import math
import random

import numpy as np
import pytest
import torch

from long_context_decoding_eta_b200 import _lib as L
from long_context_decoding_eta_b200 import synth
from long_context_decoding_eta_b200.api import EtaDecoder
from long_context_decoding_eta_b200.paged import PagedEtaDecoder, PagedKVCache

from paged_testlib import attention, rows_of

pytestmark = pytest.mark.gpu

BF16_OUT = 2.0 ** -8           # half a step of a bf16 value, relative


def make_cache(lens, Hkv, d, blk, max_pages=None, spare=5, seed=0, poison=False):
    """A cache with rows of the given lengths whose pages are scattered over the pool."""
    B = len(lens)
    nb = [-(-n // blk) for n in lens]
    max_pages = max(nb + [1]) if max_pages is None else max_pages
    n_pages = sum(nb) + spare
    c = PagedKVCache(B, Hkv, d, blk, max_pages, n_pages)
    gen = torch.Generator().manual_seed(seed)
    K = torch.randn(n_pages, Hkv, blk, d, generator=gen).to(torch.bfloat16)
    V = torch.randn(n_pages, Hkv, blk, d, generator=gen).to(torch.bfloat16)
    perm = torch.randperm(n_pages, generator=gen).int()
    k = 0
    if poison:
        K[perm[sum(nb):].long()] = float("nan")
        V[perm[sum(nb):].long()] = float("nan")
    for b, n in enumerate(lens):
        ids = perm[k:k + nb[b]]
        k += nb[b]
        c.table[b, :nb[b]] = ids.cuda()
        c.lengths[b] = n
        c.ref[ids.long().cuda()] = 1
        if poison and n % blk:
            K[int(ids[-1]), :, n % blk:] = float("nan")
            V[int(ids[-1]), :, n % blk:] = float("inf")
    c.K.copy_(K)
    c.V.copy_(V)
    return c


def check(c, q, o, lse, tau, T, blocks=None, p_eps=0.0, scale=None, gate_eps=2.0 ** -20):
    """Every head of every row against 64 bits; returns how many had no near-tie.
    blocks[b][g]: the admitted blocks (None: all)."""
    B, Hq, d = q.shape
    blk, G = c.blk, Hq // c.Hkv
    lens = c.lengths.tolist()
    table = c.table.cpu().numpy()
    q64 = q.double().cpu().numpy()
    t64 = None if tau is None else tau.double().cpu().numpy()
    K, V = (rows_of(x.double().cpu().numpy(), table, lens, blk) for x in (c.K, c.V))
    og, lg = o.double().cpu().numpy(), lse.double().cpu().numpy()
    out_eps = BF16_OUT if o.dtype == torch.bfloat16 else 2.0 ** -24
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    seen = 0
    for b in range(B):
        for h in range(Hq):
            g = h // G
            if blocks is None:
                keep = np.arange(lens[b])
            else:
                keep = np.concatenate([np.arange(j * blk, min((j + 1) * blk, lens[b]))
                                       for j in blocks[b][g]] + [np.zeros(0, dtype=int)])
            r = attention(q64[b, h], K[b][:, g], V[b][:, g], keep.astype(int),
                          None if tau is None else t64[b, h], T, scale, p_eps, out_eps,
                          gate_eps)
            o_r, lse_r, tol, ltol, tie = r
            if keep.size == 0:
                assert np.all(og[b, h] == 0) and lg[b, h] == -math.inf
                continue
            if tie:
                continue
            seen += 1
            err = np.abs(og[b, h] - o_r)
            assert np.all(err <= tol), (b, h, float((err / tol).max()))
            assert abs(lg[b, h] - lse_r) <= ltol, (b, h, lg[b, h], lse_r, ltol)
    return seen


P_EPS = {torch.bfloat16: 2.0 ** -16, torch.float32: 2.0 ** -24}


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [None, 0.0, 0.05])
@pytest.mark.parametrize("Hq,Hkv,d,blk", [(4, 1, 64, 64), (8, 8, 128, 128), (16, 2, 128, 64),
                                          (4, 2, 64, 128)])
def test_all_blocks_ragged(Hq, Hkv, d, blk, T, out):
    lens = [1, 0, 64, 65, 129, 700, 1500, 2]
    c = make_cache(lens, Hkv, d, blk, seed=Hq + d, poison=True)
    gen = torch.Generator().manual_seed(1)
    q = torch.randn(len(lens), Hq, d, generator=gen).to(torch.bfloat16).cuda()
    tau = (0.3 + 0.5 * torch.randn(len(lens), Hq, generator=gen)).cuda()
    dec = PagedEtaDecoder(c, Hq, T=T, out_dtype=out)
    o, lse = dec.decode(q, tau=tau, all_blocks=True)
    dec.check_status()
    seen = check(c, q, o, lse, None if T is None else tau, T, p_eps=P_EPS[out])
    assert seen >= 0.9 * 7 * Hq


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,prune", [(0.0, "skip"), (0.05, "skip"), (None, "skip")])
def test_block_lists(T, prune, out):
    lens = [4000, 130, 64, 0, 2999]
    Hq, Hkv, d, blk = 8, 2, 128, 64
    c = make_cache(lens, Hkv, d, blk, seed=9, poison=True)
    rng = random.Random(4)
    dec = PagedEtaDecoder(c, Hq, T=T, out_dtype=out, prune=prune)
    blocks = []
    for b, n in enumerate(lens):
        nb = -(-n // blk)
        row = [sorted(rng.sample(range(nb), rng.randint(0, nb))) for _ in range(Hkv)]
        if b == 1:
            row[0] = []                     # a head whose screen admits nothing
        for g in range(Hkv):
            dec.union_idx[b, g, :len(row[g])] = torch.tensor(row[g], dtype=torch.int32).cuda()
            dec.union_cnt[b, g] = len(row[g])
        blocks.append(row)
    gen = torch.Generator().manual_seed(2)
    q = torch.randn(len(lens), Hq, d, generator=gen).to(torch.bfloat16).cuda()
    tau = (0.3 + 0.5 * torch.randn(len(lens), Hq, generator=gen)).cuda()
    o, lse = dec.decode(q, tau=tau)
    dec.check_status()
    check(c, q, o, lse, None if T is None else tau, T, blocks, p_eps=P_EPS[out])


@pytest.mark.parametrize("cent,bound,prune", [("f32", "exact", "skip"), ("bf16", "prob", "skip"),
                                              ("f32", "prob_dim", "floor")])
def test_step_matches_the_contiguous_cache(cent, bound, prune):
    """The same tokens in a contiguous cache and behind scattered pages: metadata, lists
    and thresholds are the same bits; outputs differ by the split's third term alone."""
    w = synth.MID.with_(B=3, ctx=4096, seed=41)
    lengths = torch.tensor([4096, 3001, 64], dtype=torch.int32)
    g = {k: (v.cuda() if isinstance(v, torch.Tensor) else v)
         for k, v in synth.generate(w, "cpu", lengths=lengths).items()}
    ref = EtaDecoder(g["K"], g["V"], g["lengths"], w.Hq, w.blk, bound=bound, T=0.05, prune=prune,
                     cent_format=cent)
    ref.build_meta()
    c = PagedKVCache(w.B, w.Hkv, w.d, w.blk, w.NB, 3 * w.NB + 9)
    c.append(torch.zeros(7 * w.blk, w.Hkv, w.d, dtype=torch.bfloat16, device="cuda"),
             torch.zeros(7 * w.blk, w.Hkv, w.d, dtype=torch.bfloat16, device="cuda"),
             [0, 7 * w.blk, 7 * w.blk, 7 * w.blk])
    c.free([0])
    n1 = (lengths - 1).tolist()
    rows = [torch.cat([g[x][b, :, :n1[b]].transpose(0, 1) for b in range(3)]).contiguous()
            for x in ("K", "V")]
    c.append(rows[0], rows[1], [0] + list(np.cumsum(n1)))
    dec = PagedEtaDecoder(c, w.Hq, bound=bound, T=0.05, prune=prune, cent_format=cent)
    dec.build_meta()
    last = [torch.stack([g[x][b, :, n1[b]] for b in range(3)]) for x in ("K", "V")]
    c.append(last[0], last[1])              # the step's token: the tail refresh sees it
    bias = torch.full((w.Hq,), 1.5, device="cuda")
    o, lse = dec.step(g["q"], g["W"], bias)
    ro, rl = ref.step(g["q"], g["W"], bias)
    torch.cuda.synchronize()
    c.check_status()
    dec.check_status()
    for name in ("cent", "rmax", "var", "cnt", "tau", "head_mask", "union_cnt", "head_cnt"):
        assert torch.equal(getattr(dec, name), getattr(ref, name)), name
    if prune == "floor":
        assert torch.equal(dec.vsum, ref.vsum)
    for b in range(3):
        for h in range(w.Hkv):
            k = int(ref.union_cnt[b, h])
            assert torch.equal(dec.union_idx[b, h, :k], ref.union_idx[b, h, :k])
    # two terms against three: 2^-16 of the weights, twice, over values of up to ~4 sigma
    assert float((o - ro).abs().max()) <= 2 * 2.0 ** -16 * 5.0
    assert torch.equal(lse, rl)


def test_long_row_past_32_bit_offsets():
    """One row over a pool whose upper pages lie past 2^32 bytes (and 2^31 elements)."""
    Hkv, d, blk, n_pages = 4, 128, 128, 40000          # 5.2 GB of keys
    c = PagedKVCache(1, Hkv, d, blk, 64, n_pages)
    ids = torch.arange(n_pages - 64, n_pages, dtype=torch.int32).flip(0)
    gen = torch.Generator().manual_seed(3)
    k = torch.randn(64, Hkv, blk, d, generator=gen).to(torch.bfloat16)
    v = torch.randn(64, Hkv, blk, d, generator=gen).to(torch.bfloat16)
    c.K[ids.long().cuda()] = k.cuda()
    c.V[ids.long().cuda()] = v.cuda()
    c.table[0] = ids.cuda()
    c.lengths[0] = 64 * blk - 3
    q = torch.randn(1, 8, d, generator=gen).to(torch.bfloat16).cuda()
    dec = PagedEtaDecoder(c, 8, T=None)
    o, lse = dec.dense_decode(q)
    dec.check_status()
    small = make_cache([64 * blk - 3], Hkv, d, blk)
    small.K[small.table[0].long()] = k.cuda()
    small.V[small.table[0].long()] = v.cuda()
    assert check(small, q, o, lse, None, None, p_eps=2.0 ** -24) == 8


def test_bad_pages_and_blocks_are_skipped():
    c = make_cache([640, 300], 2, 64, 64, seed=7)
    c.table[0, 3] = -1
    c.table[0, 5] = c.n_pages
    q = torch.randn(2, 4, 64).to(torch.bfloat16).cuda()
    dec = PagedEtaDecoder(c, 4, T=None)
    o, lse = dec.dense_decode(q)
    torch.cuda.synchronize()
    assert int(dec.dev_status) == L.DEVSTAT_BAD_BLOCK
    c.table[0, 3] = c.table[0, 5] = 0       # for the oracle's gather: left out below
    blocks = [[[0, 1, 2, 4, 6, 7, 8, 9]] * 2, [list(range(5))] * 2]
    assert check(c, q, o, lse, None, None, blocks, p_eps=2.0 ** -24) == 8
    dec.dev_status.zero_()
    c.lengths[0] = 10 * 64 + 1              # past the row's capacity: clamped
    dec.dense_decode(q)
    torch.cuda.synchronize()
    assert int(dec.dev_status) & L.DEVSTAT_BAD_LENGTH


def test_meta_of_a_bad_page_is_an_empty_block():
    c = make_cache([200, 64], 1, 128, 64, seed=8)
    dec = PagedEtaDecoder(c, 4, T=0.0)
    c.table[0, 1] = c.n_pages + 3
    dec.build_meta()
    torch.cuda.synchronize()
    assert int(dec.dev_status) == L.DEVSTAT_BAD_BLOCK
    assert dec.cnt[:, 0].tolist() == [[64, 0, 64, 8], [64, 0, 0, 0]]
    assert float(dec.cent[0, 0, :, 1].abs().max()) == 0.0
    c.table[1, 0] = -5
    dec.append_update()
    torch.cuda.synchronize()
    assert dec.cnt[1, 0].tolist() == [0, 0, 0, 0]


def test_layer_refuses_wrong_tensors():
    c = make_cache([64, 64], 2, 64, 64)
    dec = PagedEtaDecoder(c, 4, T=0.0)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    tau = torch.zeros(2, 4, device="cuda")
    for bad in (q.float(), q[:1], q.cpu(), torch.zeros(2, 4, 128, device="cuda").bfloat16()[..., ::2]):
        with pytest.raises(ValueError):
            dec.decode(bad, tau=tau, all_blocks=True)
    for bad in (tau.double(), tau[:1], tau.cpu(), torch.zeros(2, 8, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            dec.decode(q, tau=bad, all_blocks=True)
    with pytest.raises(ValueError):
        dec.screen(q)
    with pytest.raises(ValueError):
        c.append(torch.zeros(3, 2, 64, device="cuda").bfloat16(),
                 torch.zeros(3, 2, 64, device="cuda").bfloat16())
    with pytest.raises(ValueError):
        c.fork([0], [1, 1])


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B", [32, 33, 257])
def test_many_rows_on_both_sides_of_the_plan_launch(B, out):
    """256 (row, KV head) pairs are laid out by the decode itself, more by a launch before it."""
    lens = [random.Random(B * 1000 + b).choice([0, 1, 63, 64, 65, 130, 200]) for b in range(B)]
    c = make_cache(lens, 8, 64, 64, seed=B, poison=True)
    gen = torch.Generator().manual_seed(B)
    q = torch.randn(B, 8, 64, generator=gen).to(torch.bfloat16).cuda()
    dec = PagedEtaDecoder(c, 8, T=None, out_dtype=out)
    o, lse = dec.decode(q, all_blocks=True)
    dec.check_status()
    assert check(c, q, o, lse, None, None, p_eps=P_EPS[out]) == 8 * sum(n > 0 for n in lens)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 1)])
def test_a_cache_with_nothing_in_it(Hq, Hkv, out):
    c = make_cache([0, 0, 0], Hkv, 128, 64, max_pages=4)
    q = torch.ones(3, Hq, 128, dtype=torch.bfloat16, device="cuda")
    dec = PagedEtaDecoder(c, Hq, T=None, out_dtype=out)
    for _ in range(2):
        o, lse = dec.decode(q, all_blocks=True)
        dec.check_status()
        assert torch.all(o == 0) and torch.all(lse == -math.inf)


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (8, 1)])
def test_a_bad_length_is_reported_and_clamped(Hq, Hkv):
    """A length below zero reads as 0, one past the table as the table's end."""
    c = make_cache([64, 256, 130], Hkv, 64, 64, max_pages=4)
    q = torch.randn(3, Hq, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    q = q.cuda()
    dec = PagedEtaDecoder(c, Hq, T=None)
    o, lse = (t.clone() for t in dec.decode(q, all_blocks=True))
    dec.check_status()
    c.lengths[0] = -3
    c.lengths[1] = 1000
    o2, lse2 = dec.decode(q, all_blocks=True)
    with pytest.raises(L.EtaError):
        dec.check_status()
    assert torch.all(o2[0] == 0) and torch.all(lse2[0] == -math.inf)
    # the same weights split among the CTAs in another way: two fp32 sums of 256 terms whose
    # weights add up to one
    assert torch.all((o2[1:] - o[1:]).abs() <= 2 * 256 * 2.0 ** -24 * c.V.abs().max().float())
