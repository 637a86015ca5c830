"""The 8-bit cache's float64 reference against facts outside itself (CPU)."""
import numpy as np
import pytest
import torch

from oracle import quant_oracle as qo


def test_e4m3_table_is_the_type_torch_has():
    bits = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(bits.double().numpy(), qo.e4m3_table())


def test_e4m3_rounding_is_torchs():
    """torch's cast rounds to nearest even; 64-bit inputs that are fp32 numbers
    take one rounding on both sides."""
    g = np.random.default_rng(0)
    x = (g.standard_normal(20000) * np.exp2(g.uniform(-12, 8, 20000))).astype(np.float32)
    x = np.clip(x, -448, 448)
    mid = (qo.e4m3_table()[:-1] + qo.e4m3_table()[1:]) / 2  # every tie
    x = np.concatenate([x, mid, -mid, [0.0]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(qo.round_e4m3(x.astype(np.float64)), want)


def test_worked_block():
    """By hand: a = 127, s = 1; 2.5 and 3.5 go to the even neighbour."""
    x = np.zeros((64, 128))
    x[0, :6] = [127, -127, 2.5, 3.5, -2.5, 0.5]
    codes, s = qo.quantise_block(x, "int8")
    assert s == 1 and list(codes[0, :6]) == [127, -127, 2, 4, -2, 0]
    x[0, 0], x[0, 1] = 448, -448
    codes, s = qo.quantise_block(x, "e4m3")
    assert s == 1 and list(codes[0, :6]) == [448, -448, 2.5, 3.5, -2.5, 0.5]
    x[0, 2], x[0, 3] = 17, 19   # steps of 2 between 16 and 32
    assert list(qo.quantise_block(x, "e4m3")[0][0, 2:4]) == [16, 20]


@pytest.mark.parametrize("code,step", [("int8", 1 / 254), ("e4m3", 1 / 16)])
def test_round_trip_bound(code, step):
    """int8: half a quantum of the block's largest value; e4m3: half a step,
    2^-4 of the value itself, or half the smallest step of the block."""
    x = np.random.default_rng(1).standard_normal((64, 128))
    codes, s = qo.quantise_block(x, code)
    y, a = codes * float(s), np.max(np.abs(x))
    bound = a * step if code == "int8" else np.maximum(np.abs(x) * step, a / 448 * 2.0 ** -10)
    assert np.all(np.abs(y - x) <= bound * (1 + 1e-6))
    assert np.max(np.abs(codes)) == qo.TOP[code]


def test_zero_and_non_finite_blocks():
    codes, s = qo.quantise_block(np.zeros((64, 128)), "int8")
    assert not codes.any() and 0 < s < 1e-30
    for bad in (np.inf, -np.inf, np.nan):
        x = np.ones((64, 128))
        x[3, 4] = bad
        codes, s = qo.quantise_block(x, "e4m3")
        assert not codes.any() and np.isnan(s)


def test_any_split_of_the_appends_stores_the_same():
    g = np.random.default_rng(2)
    k, v = g.standard_normal((2, 1, 1, 200, 128))
    ref = qo.QuantCacheOracle(1, 1, "int8")
    ref.append(k, v)
    for cuts in ([1, 63, 64, 65, 7], [199, 1], [64, 64, 72]):
        c, at = qo.QuantCacheOracle(1, 1, "int8"), 0
        for n in cuts:
            c.append(k[:, :, at:at + n], v[:, :, at:at + n])
            at += n
        for side in range(2):
            assert np.array_equal(c.values(0, 0, side), ref.values(0, 0, side))
    # the open block is exact
    assert np.array_equal(ref.values(0, 0, 0)[192:], k[0, 0, 192:])


def test_attention_is_the_loop_form():
    g = np.random.default_rng(3)
    k, v = g.standard_normal((2, 2, 2, 70, 128))
    c = qo.QuantCacheOracle(2, 2, "e4m3")
    c.append(k, v, n_new=[70, 3])
    q = g.standard_normal((2, 4, 5, 128))
    o, _, _ = c.attend(q, 0.1, n_q=[2, 5])
    for b, n, L in ((0, 2, 70), (1, 5, 3)):
        for h in range(4):
            K, V = c.values(b, h // 2, 0), c.values(b, h // 2, 1)
            for i in range(n):
                num, den = np.zeros(128), 0.0
                for j in range(L):
                    if j <= L - n + i:
                        e = np.exp(0.1 * sum(q[b, h, i, d] * K[j, d] for d in range(128)))
                        num, den = num + e * V[j], den + e
                want = num / den if den else np.zeros(128)
                assert np.allclose(o[b, h, i], want, rtol=1e-12, atol=1e-13)
    assert np.isnan(o[0, :, 2:]).all()          # not asked for
    assert not o[1, :, :2].any()                # positions -2 and -1 see nothing
