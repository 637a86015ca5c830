"""The 8-bit cache on the GPU where calls meet their limits: CTAs without
blocks, full sequences, open tokens far from their neighbours."""
import numpy as np
import pytest
import torch

from oracle import quant_oracle as qo
from tests.test_gpu_quant import SCALE, _check_values, _counts, _rows, _write

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


def _bound(oc, q, n, G, kept=None):
    """Reference, and the bound of every element of attention, of the queries
    q [Hq, n, 128] of the first sequence, which see the tokens `kept` (a mask;
    default all) up to their own places.

    u = 2^-24, w = sum p |v|, as in test_gpu_quant.py:
      2^-8 |ref| + w (2^-11 + 2 L u + 2 ds + 2^-20): o's rounding, a rounding of
      each weight to fp16, the fp32 sums, the scores' errors ds = 128 * 2^-23 *
      scale * sum |q k| + 2^-21 |score|, the roundings of rescaling.
    To fp16's floor, 2^-24 a step, half of it a rounding (calls of 17 rows and more;
    those below have a lower one):
      weights are held times 2^8 / 2^M' with 2^M' <= max p s, s = the block's scale
      or, of an open token, 2^-7 of the power of two at or under its row's
      largest |v|; they meet codes of at most 448 or 2^8 s: 2^-33 of
      max (p s) * 2^9 each, and max (p s) <= max (p t) 2^-6 with t = the
      largest |v| of the block (code 127 stands for it), or of the open row:
      L 2^-30 max (p t) in all;
      an open row's values are held with the largest in [2^7, 2^8): half a
      step is 2^-32 of the row's largest: 2^-32 sum (p t);
      an open row's keys, and q, with the largest in [2^14, 2^15): half a step
      is 2^-39 of the row's largest, in each of 128 products, on either side: ds
      grows by 128 * 2^-38 * scale * max |q| max |k of the row|.
    Nothing in it goes by tokens that the query does not see."""
    L, H = oc.length(0), oc.H
    ref, tol = np.zeros((H * G, n, 128)), np.zeros((H * G, n, 128))
    kept = np.ones(L, bool) if kept is None else kept
    full = L // 64 * 64
    for g in range(H * G):
        K, V = oc.values(0, g // G, 0), oc.values(0, g // G, 1)
        top = np.abs(V).max(1)
        for j in range(0, full, 64):
            top[j:j + 64] = top[j:j + 64].max()
        for i in range(n):
            at = np.flatnonzero(kept[:L - n + i + 1])
            if not len(at):
                continue
            k, v, t = K[at], V[at], top[at]
            s = k @ q[g, i] * SCALE
            p = np.exp(s - s.max())
            p /= p.sum()
            ds = (128 * 2.0 ** -23 * (np.abs(k) @ np.abs(q[g, i])).max() * SCALE
                  + 2.0 ** -21 * np.abs(s).max()
                  + 128 * 2.0 ** -38 * SCALE * np.abs(q[g, i]).max() * np.abs(k).max())
            ref[g, i], w = p @ v, p @ np.abs(v)
            tol[g, i] = 2.0 ** -8 * np.abs(ref[g, i]) + w * (2.0 ** -11 + 2 * L * 2.0 ** -24 + 2 * ds
                                                             + 2.0 ** -20)
            tol[g, i] += L * 2.0 ** -30 * (p * t).max() + 2.0 ** -32 * (p * t).sum()
    return ref, tol


def _attend(lrkv, cache, q):
    o = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    lrkv.quant_attn(cache, q.cuda(), SCALE, o, lrkv.quant_attn_workspace(cache, q.shape[1], q.shape[2]))
    return o.double().cpu().numpy()


# rows per KV head: each kernel and each count of copies of its rows
CALLS = [(4, 2), (4, 4), (1, 24), (2, 24), (4, 24), (4, 60)]


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("G,n", CALLS)
def test_open_tokens_far_larger_than_earlier_ones(lrkv, code, side, G, n):
    """A token that a query does not see changes nothing for it, however large
    its keys or values are; nor does one that it sees take bits from others."""
    H, L = 2, 64 + 45
    for gain in (2.0 ** 12, 2.0 ** 40, 2.0 ** 100):
        x = [_rows(1, 1, H, L), _rows(2, 1, H, L)]
        x[side][0, :, L - 2] *= gain
        x[side][0, 1, L - 1] *= 1 / gain
        cache = lrkv.QuantCache(1, H, L, code=code)
        oc = qo.QuantCacheOracle(1, H, code)
        _write(cache, oc, lrkv, *x)
        q = _rows(3, 1, H * G, n, 0.0)
        got = _attend(lrkv, cache, q)[0]
        ref, tol = _bound(oc, q[0].double().numpy(), n, G)
        # the last two see the large one: where its keys are large, as one that takes all
        # or nothing
        err = np.abs(got - ref)
        assert np.isfinite(got).all()
        assert (err <= tol)[:, :n - 2].all(), (gain, np.max((err / tol)[:, :n - 2]))
        if side:
            assert (err <= tol)[:, n - 2:].all(), (gain, np.max((err / tol)[:, n - 2:]))
        # the same bits as without the token
        cut = lrkv.QuantCache(1, H, L, code=code)
        x[side][0, :, L - 2:] = 1
        _write(cut, qo.QuantCacheOracle(1, H, code), lrkv, *x)
        assert np.array_equal(_attend(lrkv, cut, q)[0][:, :n - 2], got[:, :n - 2])
    assert cache.error() == 0


def _along(c, n, gain):
    """Keys c_t u and queries u for u of +-1: scores 128 c_t gain SCALE."""
    u = np.sign(np.random.default_rng(1).standard_normal(128))
    k = torch.from_numpy((c[:, None] * u).astype(np.float32)).to(torch.bfloat16)
    q = torch.from_numpy(np.tile(u * gain, (n, 1)).astype(np.float32)).to(torch.bfloat16)
    assert np.array_equal(k.double().numpy(), c[:, None] * u)
    return k, q


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("G,n", CALLS)
def test_scores_of_millions(lrkv, code, G, n):
    """Scores far above those at which fp32 tells two tokens from each other: the
    largest takes all, and the result is its value."""
    L = 150
    v = _rows(2, 1, 1, L)
    for sign in (1, -1):
        # a query's largest score is that of the last of these that it sees
        c = np.full(L, 0.5 if sign > 0 else -2.0)
        c[[0, 100, 140]] = [1, 2, 4] if sign > 0 else [-1, -0.5, -0.25]
        for gain in (2.0 ** 8, 2.0 ** 22, 2.0 ** 25, 2.0 ** 40, 2.0 ** 100):
            k, q = _along(c, n, gain)
            cache = lrkv.QuantCache(1, 1, L, code=code)
            oc = qo.QuantCacheOracle(1, 1, code)
            _write(cache, oc, lrkv, k[None, None], v)
            got = _attend(lrkv, cache, q[None, None].expand(1, G, n, 128).contiguous())[0]
            K, V = oc.values(0, 0, 0), oc.values(0, 0, 1)
            for i in range(n):
                pos = L - n + i
                s = np.sort(K[:pos + 1] @ q[i].double().numpy() * SCALE)
                # nothing of any other token is left: 2 ds (see _bound) away and more
                assert s[-1] - s[-2] > 2 * (128 * 2.0 ** -23 + 2.0 ** -21) * np.abs(s).max() + 200
                want = V[140 if pos >= 140 else 100 if pos >= 100 else 0]
                # o's rounding, the weight's, and the few of a sum of one term
                tol = np.abs(want) * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20)
                assert (np.abs(got[:, i] - want) <= tol).all(), (sign, gain, i)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("G,n", CALLS)
@pytest.mark.parametrize("big", [0, 70, 140])
def test_values_far_apart(lrkv, code, G, n, big):
    """A block of next to no weight with a token whose values are so much larger that
    it counts: weights of 2^-125 and more of the largest are kept whatever the values
    are."""
    L = 150
    for low, high, weight in ((-60, 60, 118), (-60, 60, 124), (-100, 20, 121), (0, 85, 90)):
        at = slice(big // 64 * 64, big // 64 * 64 + 64)
        c = np.zeros(L)
        c[at] = -1
        gain = weight * np.log(2) / (128 * SCALE)
        k, q = _along(c, n, gain)
        v = _rows(2, 1, 1, L, 0.0) * 2.0 ** low
        v[:, :, at] *= 2.0 ** -10
        v[:, :, big] = _rows(3, 1, 1, 1, 0.0)[:, :, 0] * 2.0 ** high
        cache = lrkv.QuantCache(1, 1, L, code=code)
        oc = qo.QuantCacheOracle(1, 1, code)
        _write(cache, oc, lrkv, k[None, None], v)
        q = q[None, None].expand(1, G, n, 128).contiguous()
        got = _attend(lrkv, cache, q)[0]
        ref, tol = _bound(oc, q[0].double().numpy(), n, G)
        assert (np.abs(got - ref) <= tol).all(), (low, high, weight, np.max(np.abs(got - ref) / tol))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("G,n", [(4, 1), (4, 4), (4, 8)])
def test_values_far_apart_in_long_parts(lrkv, code, G, n):
    """The same where one CTA takes all blocks of a sequence, several to a warp."""
    B, L = 200, 15 * 64 + 10
    for big, (low, high, weight) in ((0, (-60, 60, 118)), (100, (-60, 60, 124)), (600, (-100, 20, 121)),
                                     (900, (0, 85, 90)), (900, (-60, 60, 118))):
        at = slice(big // 64 * 64, big // 64 * 64 + 64)
        c = np.zeros(L)
        c[at] = -1
        k, q = _along(c, n, weight * np.log(2) / (128 * SCALE))
        v = _rows(2, 1, 1, L, 0.0) * 2.0 ** low
        v[:, :, big] = _rows(3, 1, 1, 1, 0.0)[:, :, 0] * 2.0 ** high
        oc = qo.QuantCacheOracle(1, 1, code)
        oc.append(k[None, None].double().numpy(), v.double().numpy())
        cache = lrkv.QuantCache(B, 1, L, code=code)
        lrkv.quant_append(cache, *(x.expand(B, 1, L, 128).contiguous().cuda() for x in (k, v)))
        q = q.expand(B, G, n, 128).contiguous()
        got = _attend(lrkv, cache, q)
        ref, tol = _bound(oc, q[0].double().numpy(), n, G)
        assert (np.abs(got - ref) <= tol).all(), (big, low, high, weight, np.max(np.abs(got - ref) / tol))


@pytest.mark.parametrize("G,n", CALLS)
def test_infinite_keys_of_the_open_block(lrkv, G, n):
    """An infinity among an open token's keys is the score that the formula has: of
    -inf its weight is 0, as if it were not there, +inf makes NaN.  In a full
    block it makes NaN either way."""
    H, L, at = 1, 64 + 45, 100
    x = [_rows(1, 1, H, L), _rows(2, 1, H, L)]
    oc = qo.QuantCacheOracle(1, H, "int8")
    oc.append(*(y.double().numpy() for y in x))
    x[0][0, 0, at, 7] = float("inf")
    cache = lrkv.QuantCache(1, H, 128)
    lrkv.quant_append(cache, *(y.cuda() for y in x))
    q = _rows(3, 1, H * G, n, 0.0)
    sign = torch.ones(G, n)
    sign.view(-1)[::3] = -1
    q[0, :, :, 7] = sign.to(torch.bfloat16)
    got = _attend(lrkv, cache, q)[0]
    kept = np.arange(L) != at
    ref, tol = _bound(oc, q[0].double().numpy(), n, G, kept)
    sees = (L - n + np.arange(n) >= at)[None] & (sign.numpy() > 0)
    assert np.isnan(got).all(-1)[sees].all()
    assert (np.abs(got - ref) <= tol)[~sees].all()
    # the block becomes full
    lrkv.quant_append(cache, *(_rows(5, 1, H, 19).cuda() for _ in range(2)))
    assert np.isnan(_attend(lrkv, cache, q)[0]).all()


@pytest.mark.parametrize("G,n", CALLS)
def test_scores_of_minus_infinity_alone(lrkv, G, n):
    """A query of whose tokens none counts gets 0."""
    k, v = _rows(1, 1, 1, 3), _rows(2, 1, 1, 3)
    k[..., 7] = float("-inf")
    cache = lrkv.QuantCache(1, 1, 64)
    lrkv.quant_append(cache, k.cuda(), v.cuda())
    q = _rows(3, 1, G, n, 0.0)
    q[..., 7] = 2
    assert not _attend(lrkv, cache, q).any()
    assert cache.error() == 0


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("G,n", CALLS)
def test_scores_of_millions_with_values_of_any_size(lrkv, code, G, n):
    """The exponent of the values does not get lost next to a large score."""
    L = 150
    c = np.full(L, 0.5)
    c[[0, 100, 140]] = [1, 2, 4]
    for gain in (2.0 ** 20, 2.0 ** 21, 2.0 ** 22, 2.0 ** 23, 2.0 ** 24, 2.0 ** 60):
        for size in (-60, -30, -9, -5, -3, -1, 3, 7, 40, 90):
            v = _rows(2, 1, 1, L, 0.0) * 2.0 ** size
            k, q = _along(c, n, gain)
            cache = lrkv.QuantCache(1, 1, L, code=code)
            oc = qo.QuantCacheOracle(1, 1, code)
            _write(cache, oc, lrkv, k[None, None], v)
            got = _attend(lrkv, cache, q[None, None].expand(1, G, n, 128).contiguous())[0]
            V = oc.values(0, 0, 1)
            for i in range(n):
                pos = L - n + i
                want = V[140 if pos >= 140 else 100 if pos >= 100 else 0]
                # as in test_scores_of_millions
                tol = np.abs(want) * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20)
                assert (np.abs(got[:, i] - want) <= tol).all(), (gain, size, i)


@pytest.mark.parametrize("G,n", CALLS)
@pytest.mark.parametrize("scale", [0.0, -SCALE])
def test_scales_that_are_not_positive(lrkv, G, n, scale):
    L = 64 * 3 + 45
    cache = lrkv.QuantCache(1, 2, L)
    oc = qo.QuantCacheOracle(1, 2, "int8")
    _write(cache, oc, lrkv, _rows(1, 1, 2, L), _rows(2, 1, 2, L))
    q = _rows(3, 1, 2 * G, n, 0.0)
    o = torch.zeros_like(q, device="cuda")
    lrkv.quant_attn(cache, q.cuda(), scale, o, lrkv.quant_attn_workspace(cache, 2 * G, n))
    ref, tol = _bound(oc, q[0].double().numpy() * (scale / SCALE), n, G)
    assert (np.abs(o[0].double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("G,n", CALLS)
def test_shared_queries_and_rows_of_a_wider_buffer(lrkv, G, n):
    """q with strides of 0 (one row for all heads and sequences); o's rows apart,
    what lies between them untouched."""
    B, H, L = 3, 2, 150
    cache = lrkv.QuantCache(B, H, L, code="e4m3")
    k, v = _rows(1, B, H, L), _rows(2, B, H, L)
    lrkv.quant_append(cache, k.cuda(), v.cuda())
    one = _rows(3, 1, 1, n, 0.0).cuda()
    q = one.expand(B, H * G, n, 128)
    wide = torch.full((B, n, H * G, 136), 3.0, dtype=torch.bfloat16, device="cuda")
    o = wide[..., :128].transpose(1, 2)
    ws = lrkv.quant_attn_workspace(cache, H * G, n)
    lrkv.quant_attn(cache, q, SCALE, o, ws)
    assert bool((wide[..., 128:] == 3.0).all())
    want = torch.zeros(B, H * G, n, 128, dtype=torch.bfloat16, device="cuda")
    lrkv.quant_attn(cache, q.contiguous(), SCALE, want, ws)
    assert torch.equal(o, want)
    for b in range(B):
        oc = qo.QuantCacheOracle(1, H, "e4m3")
        oc.append(k[b:b + 1].double().numpy(), v[b:b + 1].double().numpy())
        ref, tol = _bound(oc, q[b].double().cpu().numpy(), n, G)
        assert (np.abs(o[b].double().cpu().numpy() - ref) <= tol).all()
