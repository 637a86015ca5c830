"""The 8-bit cache on the GPU where calls meet their limits: CTAs without
blocks, full sequences, open tokens far from their neighbours."""
import pytest
import torch

from oracle import quant_oracle as qo
from tests.test_gpu_quant import _check_values, _counts, _rows, _write

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lrkv():
    assert torch.cuda.is_available()
    from rank_kv_cache_lrkv_b200 import lrkv as m
    return m


@pytest.mark.parametrize("n", [2, 65, 127, 190])
def test_short_ragged_appends_touch_no_block_past_the_end(lrkv, n):
    """Calls whose CTAs mostly have no block of their own.  Entries of the table
    past the last full block are out of range: a CTA that looked at one would
    set the error word."""
    B, H = 48, 4
    cache = lrkv.QuantCache(B, H, 4 * 64)
    own = cache.block_table.clone()
    n_new = [(b * 37) % (n + 1) for b in range(B)]
    n_new[0], n_new[1] = n, 0
    full = torch.tensor([x // 64 for x in n_new])[:, None]
    cache.block_table[(torch.arange(4) >= full).cuda()] = -7
    k, v, counts = _rows(1, B, H, n), _rows(2, B, H, n), _counts(n_new)
    kd, vd = k.cuda(), v.cuda()
    for _ in range(100):
        cache.seq_len.zero_()
        lrkv.quant_append(cache, kd, vd, n_new=counts)
        assert cache.seq_len.tolist() == n_new
    assert cache.error() == 0
    oc = qo.QuantCacheOracle(B, H, "int8")
    oc.append(k.double().numpy(), v.double().numpy(), n_new)
    _check_values(lrkv, cache, oc)
    # and onto open blocks, half of them full afterwards
    cache.block_table.copy_(own)
    more = [min(x, 256 - y) for x, y in zip(reversed(n_new), n_new)]
    _write(cache, oc, lrkv, _rows(3, B, H, n), _rows(4, B, H, n), more)
    _check_values(lrkv, cache, oc)
    assert cache.error() == 0


@pytest.mark.parametrize("n", [1, 2, 64, 128])
def test_tokens_for_a_full_sequence_are_reported(lrkv, n):
    """A sequence that is exactly full drops every token of the call and says
    so; its neighbour, with room or without tokens, is untouched by that."""
    B, H = 3, 2
    cache = lrkv.QuantCache(B, H, 128)
    oc = qo.QuantCacheOracle(B, H, "int8")
    _write(cache, oc, lrkv, _rows(1, B, H, 128), _rows(2, B, H, 128), [128, 0, 128])
    assert cache.error() == 0
    pages, tail = cache.pages.clone(), cache.tail.clone()
    # nothing asked of the full ones: no error
    k, v = _rows(3, B, H, n), _rows(4, B, H, n)
    _write(cache, oc, lrkv, k, v, [0, 0, -1])
    assert cache.error() == 0
    lrkv.quant_append(cache, k.cuda(), v.cuda(), n_new=_counts([n, 0, 0]))
    assert cache.error() == 3
    assert cache.seq_len.tolist() == [128, 0, 128]
    assert cache.append_counter.tolist() == [0] * B
    assert torch.equal(cache.pages, pages) and torch.equal(cache.tail, tail)
    _check_values(lrkv, cache, oc)
    # a decode step of the whole batch: the one with room takes its token
    cache.error_word.zero_()
    lrkv.quant_append(cache, k.cuda(), v.cuda())
    oc.append(k.double().numpy(), v.double().numpy(), [0, n, 0])
    assert cache.error() == 3
    _check_values(lrkv, cache, oc)
