"""The full-rank cache held in 8 bits on the GPU, against the float64 oracle.

Stored values are compared bit for bit: the codes are decided by exact
arithmetic, a scale is one fp32 division and a value one fp32 product.

Attention's bound, per element, from the formula (u = 2^-24):
  |o - ref| <= 2^-8 |ref|                       o's one rounding to bf16
             + w (2^-11 + 2 L u + 2 ds + 2^-20)  w = sum p |v|
2^-11 is one rounding of each weight to fp16, 2 L u the fp32 sums of L terms
above and below the fraction bar, ds the error of a score (it scales the
weight in both sums): 128 products added in fp32, at worst truncated,
128 * 2^-23 of scale * sum |q k|, and 2^-21 of the score itself for its
scaling and the exponential; 2^-20 for the few roundings of rescaling.

And + 2^-(25 + b) L f: fp16 has a floor.  A weight p s_v is held times 2^b /
2^M', where 2^M' <= the row's largest p s_v, b = 13 for calls of at most 16
rows a KV head and 8 above; fp16's smallest step is 2^-24, so each of L weights
is off by at most 2^-25 2^-b of the largest, times a code of at most 127 or
448: f = the largest p * (largest |v| of the token's block).  It shows where the one token that counts has code 0
in a dim, and the row's result there is what tokens of 2^-30 its weight say.

And + 2^-112 L max |v|: so does fp32.  2^(score - m) and the block's factor
2^(m + log2 s_v - M'), cut at 2^112, are separate fp32 numbers; the cut and the
flush of the first at 2^-126 only touch tokens whose p is under 2^-112, and
make their weights smaller.  It shows where a block of zeros takes p ~ 1.
"""
import numpy as np
import pytest
import torch

from oracle import quant_oracle as qo

pytestmark = pytest.mark.gpu

SCALE = 1 / np.sqrt(128)
GUARD, CANARY = 1 << 16, 0xA5


@pytest.fixture(scope="module")
def lrkv():
    assert torch.cuda.is_available()
    from rank_kv_cache_lrkv_b200 import lrkv as m
    return m


def _rows(seed, B, H, n, spread=0.5):
    g = np.random.default_rng(seed)
    x = g.standard_normal((B, H, n, 128)) * np.exp(spread * g.standard_normal((1, H, 1, 128)))
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def _order(pages):
    return torch.from_numpy(np.random.default_rng(pages).permutation(pages))


def _counts(n):
    return None if n is None else torch.tensor(n, dtype=torch.int32, device="cuda")


def _write(cache, oc, lrkv, k, v, n_new=None):
    lrkv.quant_append(cache, k.cuda(), v.cuda(), n_new=_counts(n_new))
    oc.append(k.double().numpy(), v.double().numpy(), n_new)


def _filled(lrkv, B, H, lens, code, seed=0, perm=True, extra=0, spread=0.5):
    cap = max(max(lens) + extra, 1)
    pages = B * max(1, -(-cap // 64))
    order = torch.from_numpy(np.random.default_rng(seed).permutation(pages)) if perm else None
    cache = lrkv.QuantCache(B, H, cap, code=code, page_perm=order)
    oc = qo.QuantCacheOracle(B, H, code)
    k, v = _rows(seed + 1, B, H, max(max(lens), 1), spread), _rows(seed + 2, B, H, max(max(lens), 1), spread)
    _write(cache, oc, lrkv, k, v, lens)
    return cache, oc


def _check_values(lrkv, cache, oc, dtype=torch.float32):
    B, H = oc.B, oc.H
    n = max(max(oc.length(b) for b in range(B)), 1)
    k = torch.full((B, H, n, 128), 7.0, dtype=dtype, device="cuda")
    v = torch.full_like(k, 7.0)
    lrkv.quant_read(cache, k, v)
    assert cache.seq_len.tolist() == [oc.length(b) for b in range(B)]
    assert cache.append_counter.tolist() == [0] * B
    for b in range(B):
        L = oc.length(b)
        for h in range(H):
            for side, x in enumerate((k, v)):
                want = torch.from_numpy(oc.values(b, h, side, np.float32)).to(dtype).cuda()
                assert torch.equal(torch.nan_to_num(x[b, h, :L], 5e30),
                                   torch.nan_to_num(want, 5e30)), (b, h, side)
                assert bool((x[b, h, L:] == 7.0).all())


def _check_attention(lrkv, cache, oc, G, n, n_q=None, seed=9, token_major=False, ws=None,
                     qgain=1.0):
    B, Hq = oc.B, oc.H * G
    q = (_rows(seed, B, Hq, n, 0.0) * qgain)
    qd = q.cuda()
    if token_major:
        qd = qd.transpose(1, 2).contiguous().transpose(1, 2)
    o = torch.full((B, n, Hq, 128), 3.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    if ws is None:
        ws = lrkv.quant_attn_workspace(cache, Hq, n)
    lrkv.quant_attn(cache, qd, SCALE, o, ws, n_q=_counts(n_q))
    got = o.double().cpu().numpy()
    ref, w, s2 = oc.attend(q.double().numpy(), SCALE, n_q)
    for b in range(B):
        m = n if n_q is None else min(max(n_q[b], 0), n)
        assert (got[b, :, m:] == 3.0).all()  # rows past the sequence's queries
        L = oc.length(b)
        ds = s2[b, :, :m, 0] * 128 * 2.0 ** -23 + s2[b, :, :m, 1] * 2.0 ** -21
        tol = 2.0 ** -8 * np.abs(ref[b, :, :m]) + w[b, :, :m] * (
            2.0 ** -11 + 2 * L * 2.0 ** -24 + 2 * ds + 2.0 ** -20)[..., None]
        tol += (2.0 ** (-38 if n * G <= 16 else -33) * L * s2[b, :, :m, 2]
                + 2.0 ** -112 * L * s2[b, :, :m, 3])[..., None]
        err = np.abs(got[b, :, :m] - ref[b, :, :m])
        assert not np.isnan(got[b, :, :m]).any(), b
        assert (err <= tol).all(), (b, np.max(err - tol), np.max(err / np.maximum(tol, 1e-30)))
    return o


# ------------------------------------------------------------ write and read

@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("splits", [[1], [64], [65], [200], [1] * 3 + [60, 1, 1, 130], [63, 64, 1],
                                    [37, 300, 2]])
def test_append_and_read_back(lrkv, code, splits):
    B, H = 2, 3
    cache = lrkv.QuantCache(B, H, sum(splits), code=code,
                            page_perm=_order(B * -(-sum(splits) // 64)))
    oc = qo.QuantCacheOracle(B, H, code)
    for i, n in enumerate(splits):
        _write(cache, oc, lrkv, _rows(10 * i, B, H, n), _rows(10 * i + 1, B, H, n))
    _check_values(lrkv, cache, oc)
    _check_values(lrkv, cache, oc, torch.bfloat16)
    assert cache.error() == 0


def test_pages_hold_the_documented_layout(lrkv):
    for code in ("int8", "e4m3"):
        cache, oc = _filled(lrkv, 1, 2, [130], code, seed=3)
        pages = cache.pages.cpu().numpy()
        for h in range(2):
            for j in range(2):
                slab = pages[int(cache.block_table[0, j]), h]
                scales = slab[16384:16392].view(np.float32)
                assert not slab[16392:].any()
                for side in range(2):
                    codes, s, _ = oc.stored(0, h, side)
                    assert scales[side] == s[j]
                    if side:
                        byte = slab[8192:16384].reshape(128, 64).T
                    else:
                        byte = slab[:8192].reshape(64, 8, 16).copy()
                        byte[1::2] = byte[1::2][:, [4, 5, 6, 7, 0, 1, 2, 3]]
                        byte = byte.reshape(64, 128)
                    byte = np.ascontiguousarray(byte)
                    got = byte.astype(np.int64) - 128 if code == "int8" else \
                        torch.from_numpy(byte).view(torch.float8_e4m3fn).double().numpy()
                    assert np.array_equal(got, codes[64 * j:64 * j + 64])
        # the open block's rows, exactly
        tail = cache.tail[0, 1, :, :2].double().cpu().numpy()
        for side in range(2):
            assert np.array_equal(tail[side], oc.rows[0][1][side][128:])


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_ragged_appends_and_ranges(lrkv, code):
    B, H = 5, 2
    cache = lrkv.QuantCache(B, H, 400, code=code)
    oc = qo.QuantCacheOracle(B, H, code)
    for i, n_new in enumerate(([0, 1, 63, 64, 150], [70, -3, 1, 500, 149], [1, 1, 1, 1, 1])):
        _write(cache, oc, lrkv, _rows(i, B, H, 150), _rows(i + 50, B, H, 150), n_new)
    _check_values(lrkv, cache, oc)
    # token ranges that start before the cache, inside blocks and past the end
    first = [-5, 60, 64, 213, 400]
    for n in (1, 5, 64, 131):
        k = torch.full((B, n, H, 128), 2.0, device="cuda").transpose(1, 2)
        v = k.clone()
        lrkv.quant_read(cache, k, v, first=_counts(first))
        for b in range(B):
            for side, x in enumerate((k, v)):
                for h in range(H):
                    want = np.full((n, 128), 2.0, np.float32)
                    vals = oc.values(b, h, side, np.float32)
                    for i in range(n):
                        if 0 <= first[b] + i < len(vals):
                            want[i] = vals[first[b] + i]
                    assert np.array_equal(x[b, h].cpu().numpy(), want), (n, b, h, side)


def test_read_of_more_tokens_than_there_can_be(lrkv):
    """Rows of tokens that do not exist are not written, so n may be anything."""
    lens = [150, 0, 64]
    cache, oc = _filled(lrkv, 3, 2, lens, "int8", extra=100)
    first = [100, -7, 0]
    k = torch.full((3, 2, 160, 128), 2.0, device="cuda")
    v = k.clone()
    lrkv._quant_call("lrkv_quant_read", cache, None, _counts(first).data_ptr(), 2 ** 31 - 1,
                     k.data_ptr(), v.data_ptr(), lrkv.LRKV_F32, *k.stride()[:3])
    for b in range(3):
        for h in range(2):
            for side, x in enumerate((k, v)):
                want = np.full((160, 128), 2.0, np.float32)
                vals = oc.values(b, h, side, np.float32)[max(first[b], 0):]
                want[:len(vals)] = vals
                assert np.array_equal(x[b, h].cpu().numpy(), want), (b, h, side)


def test_read_into_rows_of_every_alignment(lrkv):
    """fp32 rows 16 bytes past a 32-byte border, by pointer and by stride."""
    cache, oc = _filled(lrkv, 1, 2, [150], "int8")
    for shift, row in ((0, 128), (4, 128), (0, 132), (4, 136)):
        buf = torch.full((2, 2 * 150 * row + 64), 2.0, device="cuda")
        k, v = (x[shift:shift + 2 * 150 * row].view(1, 2, 150, row)[..., :128] for x in buf)
        lrkv.quant_read(cache, k, v)
        for h in range(2):
            for side, x in enumerate((k, v)):
                assert np.array_equal(x[0, h].cpu().numpy(), oc.values(0, h, side, np.float32))
        assert int((buf == 2.0).sum()) >= 2 * (64 + 2 * 150 * (row - 128))


def test_strided_inputs(lrkv):
    """k and v as slices of one fused projection [B, n, (H k, H v), 128]."""
    B, H, n = 2, 3, 77
    x = _rows(1, B, 2 * H, n).transpose(1, 2).contiguous()
    cache = lrkv.QuantCache(B, H, n)
    oc = qo.QuantCacheOracle(B, H, "int8")
    xd = x.cuda().transpose(1, 2)
    lrkv.quant_append(cache, xd[:, :H], xd[:, H:])
    xt = x.transpose(1, 2).double().numpy()
    oc.append(xt[:, :H], xt[:, H:])
    _check_values(lrkv, cache, oc)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_extreme_values(lrkv, code):
    """Zeros, the smallest and largest bf16 numbers, exact ties, and blocks
    with an infinity or a NaN (they read as NaN, their neighbours do not)."""
    g = np.random.default_rng(5)
    x = torch.zeros(1, 7, 192, 128, dtype=torch.bfloat16)
    big = torch.finfo(torch.bfloat16).max
    x[0, 1] = torch.from_numpy(g.uniform(-1, 1, (192, 128))).to(torch.bfloat16) * big
    x[0, 2] = torch.from_numpy(g.standard_normal((192, 128)) * 2.0 ** -125).to(torch.bfloat16)
    # every bf16 number of three binades under 127 and 254: ties among them
    grid = torch.arange(0, 384, 0.5).to(torch.bfloat16)
    x[0, 3].view(-1)[:768] = torch.where(grid <= 127, grid, 0)
    x[0, 3, 0, 1] = 127
    x[0, 4, :64].view(-1)[:768] = torch.where(grid <= 254, grid, 0)
    x[0, 4, 0, 1] = 254
    x[0, 4, 64:128].view(-1)[:768] = grid / 384 * 448
    x[0, 4, 64, 1] = 448
    x[0, 5] = torch.from_numpy(g.standard_normal((192, 128))).to(torch.bfloat16)
    x[0, 5, 70, 3] = float("inf")
    x[0, 5, 191, 127] = float("nan")
    x[0, 6] = torch.from_numpy(np.exp(g.uniform(-80, 80, (192, 128)))).to(torch.bfloat16)
    v = x.flip(1).contiguous()
    cache = lrkv.QuantCache(1, 7, 192, code=code)
    oc = qo.QuantCacheOracle(1, 7, code)
    _write(cache, oc, lrkv, x, v)
    _check_values(lrkv, cache, oc)


def test_setting_the_length_back(lrkv):
    """Rejected drafts: seq_len goes back by up to 64 tokens, across a block
    that was already quantised, and other tokens follow."""
    for code in ("int8", "e4m3"):
        B, H = 2, 2
        cache, oc = _filled(lrkv, B, H, [100, 130], code, extra=200)
        for i, (n, back) in enumerate(((64, 64), (30, 29), (50, 50), (1, 1), (70, 64), (3, 0))):
            _write(cache, oc, lrkv, _rows(20 + i, B, H, n), _rows(40 + i, B, H, n))
            cache.seq_len -= back
            for b in range(B):
                oc.truncate(b, oc.length(b) - back)
            _check_values(lrkv, cache, oc)
            _check_attention(lrkv, cache, oc, 2, 3)


def test_appends_past_the_capacity_are_dropped(lrkv):
    cache, oc = _filled(lrkv, 2, 2, [120, 20], "int8", perm=False)
    assert cache.max_pages == 2
    before = cache.pages.clone()
    k, v = _rows(1, 2, 2, 30), _rows(2, 2, 2, 30)
    lrkv.quant_append(cache, k.cuda(), v.cuda())
    assert cache.error() == 3 and cache.seq_len.tolist() == [128, 50]
    oc.append(k.double().numpy(), v.double().numpy(), [8, 30])
    _check_values(lrkv, cache, oc)
    assert torch.equal(cache.pages[0], before[0])


def _guard(lrkv, cache):
    """Move the cache's buffers between bands of a known byte."""
    bufs = []
    for name, field in (("pages", "pages"), ("tail", "tail")):
        t = getattr(cache, name)
        n = t.numel() * t.element_size()
        buf = torch.full((2 * GUARD + n,), CANARY, dtype=torch.uint8, device="cuda")
        view = buf[GUARD:GUARD + n].view(t.dtype).view(t.shape)
        view.zero_()
        setattr(cache, name, view)
        setattr(cache.desc, field, view.data_ptr())
        bufs.append(buf)
    return bufs


def test_bad_pages_are_skipped_and_reported(lrkv):
    B, H = 2, 2
    k, v = _rows(1, B, H, 300), _rows(2, B, H, 300)
    for bad in (-1, 2 ** 31 - 1, B * 5):
        cache = lrkv.QuantCache(B, H, 300)
        bands = _guard(lrkv, cache)
        cache.block_table[0, 1] = bad
        oc = qo.QuantCacheOracle(B, H, "int8")
        _write(cache, oc, lrkv, k, v)
        assert cache.error() == 2
        out = [torch.full((B, H, 300, 128), 7.0, device="cuda") for _ in range(2)]
        lrkv.quant_read(cache, *out)
        for b in range(B):
            for h in range(H):
                for side in range(2):
                    want = oc.values(b, h, side, np.float32)
                    if b == 0:
                        want[64:128] = 0
                    assert np.array_equal(out[side][b, h].cpu().numpy(), want)
        # attention leaves the block's tokens out: the oracle without them
        q = _rows(3, B, H * 2, 2)
        o = torch.zeros(B, H * 2, 2, 128, dtype=torch.bfloat16, device="cuda")
        cache.error_word.zero_()
        lrkv.quant_attn(cache, q.cuda(), SCALE, o, lrkv.quant_attn_workspace(cache, H * 2, 2))
        assert cache.error() == 2
        for h in range(H * 2):
            K, V = oc.values(0, h // 2, 0), oc.values(0, h // 2, 1)
            keep = np.r_[0:64, 128:300]
            for i in range(2):
                kk = keep[keep <= 298 + i]
                s = K[kk] @ q[0, h, i].double().numpy() * SCALE
                p = np.exp(s - s.max())
                ref = p @ V[kk] / p.sum()
                assert np.abs(o[0, h, i].double().cpu().numpy() - ref).max() < 2e-2
        for buf in bands:
            assert bool((buf[:GUARD] == CANARY).all() and (buf[-GUARD:] == CANARY).all())


def test_pages_beyond_four_gigabytes(lrkv):
    """Sequences at the far end of a pool whose byte offsets pass 32 bits."""
    B, H = 2, 8
    cache, oc = _filled(lrkv, B, H, [200, 129], "int8", perm=False)
    pages = (9 << 29) // (H * lrkv.QUANT_SLAB_BYTES)
    big = torch.zeros((pages, H, lrkv.QUANT_SLAB_BYTES), dtype=torch.uint8, device="cuda")
    ids = torch.tensor([[pages - 1, 0, pages - 3, pages // 2], [5, pages - 2, 9, 11]],
                       dtype=torch.int32, device="cuda")
    cache.pages, cache.block_table = big, ids
    cache.desc.pages, cache.desc.num_pages = big.data_ptr(), pages
    cache.desc.block_table = ids.data_ptr()
    cache.seq_len.zero_()
    k, v = _rows(1, B, H, 200), _rows(2, B, H, 200)
    lrkv.quant_append(cache, k.cuda(), v.cuda(), n_new=_counts([200, 129]))
    _check_values(lrkv, cache, oc)
    _check_attention(lrkv, cache, oc, 2, 1)
    _check_attention(lrkv, cache, oc, 4, 40)
    assert cache.error() == 0


# ----------------------------------------------------------------- attention

@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("B,H,G,lens,n,n_q", [
    (1, 1, 1, [1], 1, None),
    (1, 2, 4, [63], 1, None),
    (2, 2, 4, [64, 65], 1, None),
    (3, 2, 2, [0, 700, 129], 1, None),                    # an empty sequence
    (2, 3, 8, [500, 191], 1, None),
    (1, 1, 5, [333], 1, None),                            # an odd ratio
    (1, 1, 64, [200], 1, None),                           # one KV head for all
    (2, 2, 4, [300, 128], 4, None),                       # drafted tokens
    (3, 1, 3, [70, 5, 0], 7, [7, 9, 2]),                  # more queries than tokens
    (2, 2, 1, [257, 64], 64, [64, 0]),
    (2, 1, 4, [200, 200], 50, [1, 50]),
    (1, 2, 4, [130], 130, None),                          # a whole prompt
    (2, 2, 2, [515, 300], 300, [260, 300]),
    (1, 1, 7, [400], 111, None),
    (1, 1, 128, [150], 9, None),
])
def test_attention(lrkv, code, B, H, G, lens, n, n_q):
    cache, oc = _filled(lrkv, B, H, lens, code, seed=B + n)
    _check_attention(lrkv, cache, oc, G, n, n_q, token_major=n > 4)
    assert cache.error() == 0


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("n", [1, 40])
def test_attention_with_sharp_scores_and_uneven_blocks(lrkv, code, n):
    """Scores of a hundred, block scales 2^30 apart, blocks of zeros."""
    B, H, L = 2, 2, 400
    k, v = _rows(1, B, H, L), _rows(2, B, H, L)
    v[:, :, 64:128] *= 2.0 ** -30
    v[:, :, 128:192] *= 2.0 ** 18
    v[:, :, 192:256] = 0
    k[:, :, 256:320] *= 2.0 ** -20
    k[:, 1, 0:64] = 0
    cache = lrkv.QuantCache(B, H, L, code=code)
    oc = qo.QuantCacheOracle(B, H, code)
    _write(cache, oc, lrkv, k, v, [L, 330])
    _check_attention(lrkv, cache, oc, 4, n)
    _check_attention(lrkv, cache, oc, 4, n, qgain=32.0)


def test_blocks_of_nan_show_where_they_are_seen(lrkv):
    """A NaN block makes NaN of every query that sees it and of no other."""
    B, H, L, n = 1, 2, 300, 200
    for side in range(2):
        x = [_rows(1, B, H, L), _rows(2, B, H, L)]
        x[side][0, 0, 130, 7] = float("nan")
        cache = lrkv.QuantCache(B, H, L)
        lrkv.quant_append(cache, x[0].cuda(), x[1].cuda())
        for n in (1, 200):
            q = _rows(3, B, 4, n).cuda()
            o = torch.zeros_like(q)
            lrkv.quant_attn(cache, q, SCALE, o, lrkv.quant_attn_workspace(cache, 4, n))
            nan = torch.isnan(o)
            assert not nan[0, 2:].any()
            for i in range(n):
                assert bool(nan[0, :2, i].all() if L - n + i >= 128 else not nan[0, :2, i].any())


def test_open_tokens_that_are_not_finite(lrkv):
    """An open token's NaN or infinity among its values, or a NaN among its
    keys, makes NaN of the queries that see it; earlier ones stay exact."""
    B, H, L, n = 1, 2, 150, 24
    clean, oc = _filled(lrkv, B, H, [L], "int8", seed=0, perm=False)
    q = _rows(3, B, 4, n).cuda()
    ref, _, _ = oc.attend(q.double().cpu().numpy(), SCALE)
    for side, what in ((0, "nan"), (1, "nan"), (1, "inf")):
        x = [_rows(1, B, H, L), _rows(2, B, H, L)]
        x[side][0, 0, 140, 7] = float(what)
        cache = lrkv.QuantCache(B, H, L)
        lrkv.quant_append(cache, x[0].cuda(), x[1].cuda())
        for m in (n, 2, 12):   # the last m queries, in calls of either kind
            qm = q[:, :, n - m:].contiguous()
            o = torch.zeros_like(qm)
            lrkv.quant_attn(cache, qm, SCALE, o, lrkv.quant_attn_workspace(cache, 4, m))
            for i in range(m):
                sees = L - m + i >= 140
                assert bool(torch.isnan(o[0, :2, i]).all()) == sees, (side, what, m, i)
                assert not torch.isnan(o[0, 2:, i]).any()
                for h in range(4):
                    if h >= 2 or not sees:
                        err = np.abs(o[0, h, i].double().cpu().numpy() - ref[0, h, n - m + i])
                        assert err.max() < 2e-2


def test_garbage_past_the_end_does_not_count(lrkv):
    """NaN in pages, tail slots and block-table entries that no token uses."""
    for n in (1, 40):
        cache, oc = _filled(lrkv, 2, 2, [100, 64], "e4m3", extra=300)
        used = cache.block_table[:, 0].tolist() + cache.block_table[0, 1:1].tolist()
        mask = torch.ones(cache.num_pages, dtype=torch.bool)
        mask[used] = False
        cache.pages[mask.cuda()] = 0xFF
        cache.tail[0, :, :, 100:] = float("nan")
        cache.tail[0, :, :, :36] = float("inf")
        cache.tail[1] = float("nan")
        cache.block_table[0, 1:] = -7   # the open block needs no page
        cache.block_table[1, 1:] = 1 << 30
        _check_attention(lrkv, cache, oc, 4, n)
        assert cache.error() == 0


def test_non_finite_queries(lrkv):
    """A row's infinity or NaN stays in that row."""
    for n in (1, 40):
        cache, oc = _filled(lrkv, 1, 1, [200], "int8")
        q = _rows(4, 1, 4, n)
        q[0, 1, 0, 5] = float("nan")
        q[0, 2, n - 1, 9] = float("inf")
        o = torch.zeros(1, 4, n, 128, dtype=torch.bfloat16, device="cuda")
        lrkv.quant_attn(cache, q.cuda(), SCALE, o, lrkv.quant_attn_workspace(cache, 4, n))
        bad = torch.isnan(o).all(-1)[0].cpu()
        want = torch.zeros(4, n, dtype=torch.bool)
        want[1, 0] = want[2, n - 1] = True
        assert torch.equal(bad, want)
        assert not torch.isnan(o).any(-1)[0].cpu()[~want].any()


@pytest.mark.parametrize("lens,G,n", [([4000, 3001], 4, 300), ([700, 64, 2500], 3, 260),
                                      ([5000], 8, 16), ([3000, 129], 2, 40), ([9000, 10], 4, 4)])
def test_long_calls_over_many_ranges(lrkv, lens, G, n):
    """Units of many parts and CTAs of many units: every call, one after the
    other, against the formula in 64 bits on the GPU."""
    B, H = len(lens), 2
    cache, _ = _filled(lrkv, B, H, lens, "int8")
    L = max(lens)
    k, v = (torch.zeros(B, H, L, 128, device="cuda") for _ in range(2))
    lrkv.quant_read(cache, k, v)
    q = _rows(4, B, H * G, n).cuda()
    s = (q.double().view(B, H, G * n, 128) @ k.double().transpose(2, 3) * SCALE).view(B, H, G, n, L)
    at = torch.tensor(lens, device="cuda")[:, None] - n + torch.arange(n, device="cuda")
    seen = torch.arange(L, device="cuda") <= at[..., None]
    p = torch.softmax(s.masked_fill(~seen[:, None, None], -1e300), -1) * seen.any(-1)[:, None, None, :, None]
    ref = (p.view(B, H, G * n, L) @ v.double()).view(B, H * G, n, 128)
    w = (p.view(B, H, G * n, L) @ v.double().abs()).view(B, H * G, n, 128)
    # the bound above with ds <= 2^-10 (sum |q k| scale < 60 here) and its
    # floors left out (no block is far from its neighbours)
    tol = 2.0 ** -8 * ref.abs() + w * (2.0 ** -11 + 2 * L * 2.0 ** -24 + 2.0 ** -9)
    ws = lrkv.quant_attn_workspace(cache, H * G, n)
    first = None
    for _ in range(6):
        o = torch.zeros_like(q)
        lrkv.quant_attn(cache, q, SCALE, o, ws)
        assert bool(((o.double() - ref).abs() <= tol).all())
        assert first is None or torch.equal(first, o)
        first = o
    assert cache.error() == 0


@pytest.mark.parametrize("L,G,n", [(20000, 8, 1), (20000, 8, 2), (9001, 1, 1), (700, 5, 3)])
def test_the_only_head_of_a_sequence(lrkv, L, G, n):
    """One unit over many CTAs: its parts are added up by the last of them."""
    cache, oc = _filled(lrkv, 1, 1, [L], "int8", seed=G)
    ws = lrkv.quant_attn_workspace(cache, G, n)
    first = _check_attention(lrkv, cache, oc, G, n, ws=ws)
    for _ in range(4):
        assert torch.equal(first, _check_attention(lrkv, cache, oc, G, n, ws=ws))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("G,n", [(1, 17), (1, 33), (3, 11), (5, 13), (7, 5), (33, 2), (127, 1), (1, 129),
                                 (3, 100), (5, 52), (100, 3)])
def test_group_sizes_of_many_rows(lrkv, code, G, n):
    """Rows that are no power of two, in one tile and in several."""
    cache, oc = _filled(lrkv, 3, 2, [200, 64, 331], code, seed=G)
    _check_attention(lrkv, cache, oc, G, n, [n, n // 2, n], seed=n)
    assert cache.error() == 0


@pytest.mark.parametrize("B", [400, 1024])
@pytest.mark.parametrize("G,n", [(2, 1), (4, 3), (1, 20), (2, 60), (1, 130)])
def test_large_batches(lrkv, B, G, n):
    """The tables of lengths take shared memory from the pages in flight."""
    g = np.random.default_rng(B + n)
    lens = g.integers(0, 150, B).tolist()
    lens[0], lens[-1] = 0, 200
    n_q = [int(x) if i % 7 == 0 or i == B - 1 else 0 for i, x in enumerate(g.integers(0, n + 1, B))]
    n_q[-1] = n
    cache, oc = _filled(lrkv, B, 1, lens, "int8", seed=n)
    _check_attention(lrkv, cache, oc, G, n, n_q)
    assert cache.error() == 0


@pytest.mark.parametrize("n", [1, 5, 100])
def test_the_same_call_gives_the_same_bits(lrkv, n):
    cache, oc = _filled(lrkv, 3, 2, [900, 64, 2000], "int8")
    q = _rows(4, 3, 8, n).cuda()
    ws = lrkv.quant_attn_workspace(cache, 8, n)
    o = [torch.zeros_like(q) for _ in range(8)]
    for x in o:
        lrkv.quant_attn(cache, q, SCALE, x, ws)
    assert all(torch.equal(o[0], x) for x in o[1:])


def test_a_large_workspace_serves_smaller_calls(lrkv):
    cache, oc = _filled(lrkv, 2, 2, [300, 130], "int8")
    ws = lrkv.quant_attn_workspace(cache, 8, 64)
    for n in (64, 1, 17, 64, 3):
        _check_attention(lrkv, cache, oc, 4, n, ws=ws, seed=n)


def test_short_workspace_is_refused(lrkv):
    cache, _ = _filled(lrkv, 2, 2, [300, 130], "int8")
    q = _rows(1, 2, 8, 4).cuda()
    o = torch.full_like(q, 3.0)
    ws = lrkv.quant_attn_workspace(cache, 8, 4)
    with pytest.raises(lrkv.LrkvError) as e:
        lrkv.quant_attn(cache, q, SCALE, o, ws[:-16])
    assert e.value.status == -4
    torch.cuda.synchronize()
    assert bool((o == 3.0).all())


def test_two_streams_at_once(lrkv):
    """Two caches, each with its own workspace, on streams of their own."""
    pairs = [_filled(lrkv, 2, 2, [1500, 700], code, seed=s) for s, code in ((0, "int8"), (5, "e4m3"))]
    q = [_rows(s, 2, 8, 1).cuda() for s in (1, 2)]
    ws = [lrkv.quant_attn_workspace(c, 8, 1) for c, _ in pairs]
    want = []
    for (c, _), x, w in zip(pairs, q, ws):
        want.append(lrkv.quant_attn(c, x, SCALE, torch.zeros_like(x), w))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[torch.zeros_like(x) for _ in range(20)] for x in q]
    for r in range(20):
        for i in range(2):
            lrkv.quant_attn(pairs[i][0], q[i], SCALE, got[i][r], ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(want[i], x) for x in got[i])


# ------------------------------------------------------- the calls together

@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_prompt_then_generation(lrkv, code):
    """A prompt in two chunks, attended as it comes in, then single tokens
    across a block's end, then drafted tokens of which some are rejected."""
    B, H, G = 2, 2, 4
    cache = lrkv.QuantCache(B, H, 400, code=code, page_perm=_order(14))
    oc = qo.QuantCacheOracle(B, H, code)
    ws = lrkv.quant_attn_workspace(cache, H * G, 150)
    for i, n in enumerate((150, 37)):
        _write(cache, oc, lrkv, _rows(i, B, H, n), _rows(i + 5, B, H, n))
        _check_attention(lrkv, cache, oc, G, n, ws=ws, seed=i)
    for i in range(8):
        _write(cache, oc, lrkv, _rows(20 + i, B, H, 1), _rows(40 + i, B, H, 1))
        _check_attention(lrkv, cache, oc, G, 1, ws=ws, seed=60 + i)
    _write(cache, oc, lrkv, _rows(80, B, H, 5), _rows(81, B, H, 5), [5, 4])
    _check_attention(lrkv, cache, oc, G, 5, [5, 4], ws=ws, seed=82)
    cache.seq_len -= 3
    for b in range(B):
        oc.truncate(b, oc.length(b) - 3)
    _write(cache, oc, lrkv, _rows(83, B, H, 1), _rows(84, B, H, 1))
    _check_attention(lrkv, cache, oc, G, 1, ws=ws, seed=85)
    _check_values(lrkv, cache, oc)
    assert cache.error() == 0


def test_captured_step_replays(lrkv):
    """Append, attend and read back in one graph, replayed over a block's end;
    the graph reads lengths and rows from the device each time."""
    B, H, G = 2, 2, 4
    cache, oc = _filled(lrkv, B, H, [60, 125], "int8", extra=80)
    k = torch.zeros(B, H, 1, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    q = torch.zeros(B, H * G, 128, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros_like(q)
    out = [torch.zeros(B, H, 256, 128, device="cuda") for _ in range(2)]
    ws = lrkv.quant_attn_workspace(cache, H * G, 1)
    keep = cache.seq_len.clone()

    def step():
        lrkv.quant_append(cache, k, v)
        lrkv.quant_attn(cache, q, SCALE, o, ws)
        lrkv.quant_read(cache, *out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    cache.seq_len.copy_(keep)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    cache.seq_len.copy_(keep)
    for i in range(10):
        kk, vv, qq = _rows(i, B, H, 1), _rows(i + 20, B, H, 1), _rows(i + 40, B, H * G, 1)
        k.copy_(kk), v.copy_(vv), q.copy_(qq[:, :, 0])
        graph.replay()
        oc.append(kk.double().numpy(), vv.double().numpy())
        ref, w, _ = oc.attend(qq.double().numpy(), SCALE)
        err = np.abs(o.double().cpu().numpy() - ref[:, :, 0])
        assert (err <= 2.0 ** -8 * np.abs(ref[:, :, 0]) + 2.0 ** -10 * w[:, :, 0]).all()
        for b in range(B):
            L = oc.length(b)
            assert np.array_equal(out[0][b, 1, :L].cpu().numpy(), oc.values(b, 1, 0, np.float32))
    assert cache.error() == 0
