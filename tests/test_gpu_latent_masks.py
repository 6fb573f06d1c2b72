"""GPU: what a latent call must not depend on or let through."""
import pytest
import torch

from tests.test_gpu_latent import KINDS, _attend, _cache, _pages

pytestmark = pytest.mark.gpu


def test_the_same_call_gives_the_same_bits():
    # the sums' order is fixed: what a call gives does not depend on timing
    lens, nb, L = [2500, 700, 1300], 300, 512
    for kind, token in KINDS:
        cache, scale, sc = _cache(45, nb, L, kind, token)
        cache, sc = cache.cuda(), None if sc is None else sc.cuda()
        bt = _pages(45, lens, 160, nb)
        q = torch.randn(3, 1, 128, L + 64, generator=torch.Generator().manual_seed(46)).to(torch.bfloat16)
        q = (q * 3).cuda()
        first = _attend(q, cache, bt, lens, L, scale, sc, kind, 0.07)
        for _ in range(100):
            assert torch.equal(_attend(q, cache, bt, lens, L, scale, sc, kind, 0.07), first)
