"""Page operations on both sides of the sizes where another kernel takes over, against the
plain model of the rules."""
import random

import pytest
import torch

from long_context_decoding_eta_b200 import _lib as L
from long_context_decoding_eta_b200.paged import PagedKVCache

from test_gpu_pages import Both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 63, 64, 65, 150])
def test_forks_of_few_and_many_pairs(n):
    """64 pairs are planned by every CTA, more by a launch before; refused pairs among them."""
    t = Both(320, 1, 64, 64, 3, 700, seed=n)
    rng = random.Random(n)
    t.append([rng.choice([0, 1, 64, 100, 128, 150]) for _ in range(160)] + [0] * 160)
    src, dst = [rng.randrange(160) for _ in range(n)], rng.sample(range(160, 320), n)
    t.fork(src, dst)
    t.check()
    t.free(dst)
    if n > 4:
        dst[1], dst[2], src[3], dst[4] = dst[0], 320, -1, next(
            b for b in range(160) if t.m.len[b])      # named before, out of range, not empty
        t.fork(src, dst)
        t.check(L.DEVSTAT_BAD_ROW)


@pytest.mark.parametrize("n", [64, 65])
def test_forks_while_pages_last(n):
    t = Both(2 * n, 1, 64, 64, 2, n + 20, seed=n)
    t.append([70] * 10 + [0] * (2 * n - 10))          # 20 pages; n left, then n - 40
    t.append([0] * 10 + [1] * 40 + [0] * (2 * n - 50))
    t.fork([i % 10 for i in range(n)], list(range(n, 2 * n)))
    t.check(L.DEVSTAT_NO_PAGE)
    assert sum(x > 0 for x in t.m.len[n:]) == n - 40


@pytest.mark.parametrize("n", [1024, 1025])
def test_copies_on_both_sides_of_128_mb(n):
    """1,024 pairs of 128 KB pages are checked by every copying CTA, 1,025 by a launch
    before; refused pairs among them."""
    n_pages = 2 * n + 5
    c = PagedKVCache(1, 4, 128, 64, 1, n_pages)
    gen = torch.Generator(device="cuda").manual_seed(n)
    for x in (c.K, c.V):
        x.normal_(generator=gen)
    K, V = c.K.clone(), c.V.clone()
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(n))
    src, dst = perm[:n].clone(), perm[n:2 * n].clone()
    dst[n - 1], dst[5], dst[7], src[9] = dst[0], src[3], -1, n_pages
    ok = torch.ones(n, dtype=torch.bool)
    ok[[n - 1, 5, 7, 9]] = False
    c.copy_pages(src, dst)
    f, t = src[ok].cuda(), dst[ok].cuda()
    K[t], V[t] = K[f], V[f]
    torch.cuda.synchronize()
    assert int(c.dev_status) == L.DEVSTAT_BAD_ROW
    assert torch.equal(c.K, K) and torch.equal(c.V, V)
