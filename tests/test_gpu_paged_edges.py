"""Calls at the edges of what the paged decodes take: shares without a single key, values
that are not finite, thresholds and temperatures at the ends of their range, index lists."""
import math

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
