"""Pins of the 8-bit cache's and the adjusted logits' oracle."""
import numpy as np
import pytest
import torch

from oracle import quant as oq


def test_codes_against_torch():
    """All 256 values, and the rounding of a sweep over the range, ties among it."""
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(oq.VALUES, want, equal_nan=True)
    mid = (oq.VALUES[:126] + oq.VALUES[1:127]) / 2
    x = np.concatenate([mid, oq.VALUES[:127], np.random.default_rng(0).normal(size=5000) * 100,
                        np.random.default_rng(1).normal(size=5000) * 0.01]).clip(-448, 448)
    x = np.concatenate([x, -x])
    got = torch.from_numpy(oq.encode(x)).view(torch.float8_e4m3fn).to(torch.float64)
    assert torch.equal(got, torch.from_numpy(x).to(torch.float32).to(torch.float8_e4m3fn).to(torch.float64))


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.5, 1), (1.0, -8), (1.75, -8), (1.8, -7), (0.0, -127), (1e-45, -127),
                                   (3e38, 120)])
def test_exponent(top, e):
    assert oq.exponent(top) == e


def test_append_keeps_earlier_tokens_and_forgets_void_ones():
    rng = np.random.default_rng(2)
    table = np.array([[1, 0]], dtype=np.int32)
    codes = np.zeros((2, 1, 16, 4), dtype=np.uint8)
    scale = np.full((2, 1, 1), 200, dtype=np.uint8)
    x = rng.normal(size=(5, 1, 4))
    ck, cv, sk, sv, ek, _ = oq.append(codes, codes, scale, scale, table, [0, 5], [0], x, x, 0.0)
    assert sk[1, 0, 0] < 200 and sk[0, 0, 0] == 200          # a block that begins anew; one not reached
    before = oq.held(ck, sk)[1, 0, :5]
    assert np.all(np.abs(before - x[:, 0]) <= 2.0 ** -4 * np.abs(x[:, 0]) + 2.0 ** (int(sk[1, 0, 0]) - 137))
    # a larger token: earlier ones keep their values (but for subnormals)
    ck, cv, sk, sv, _, _ = oq.append(ck, cv, sk, sv, table, [0, 1], [5], 100 * x[:1], x[:1], 0.0)
    after = oq.held(ck, sk)[1, 0, :5]
    assert np.all(np.abs(after - before) <= 2.0 ** (int(sk[1, 0, 0]) - 137))
    # taken back: from slot 3 on the block is void, its scale stays
    ck2, _, sk2, _, _, _ = oq.append(ck, cv, sk, sv, table, [0, 1], [3], x[:1], x[:1], 0.0)
    assert sk2[1, 0, 0] == sk[1, 0, 0] and np.array_equal(ck2[1, 0, :3], ck[1, 0, :3])


def test_adjust_by_hand():
    x = np.array([[2.0, -2.0, 1.0, 0.5, 4.0]] * 3)
    kw = dict(history=[[0, 1, 2, 2]], prompt_len=[2], repetition=[2.0], frequency=[0.25], presence=[0.5])
    out, _ = oq.adjust(x, [0, 1], **kw)
    assert out[0].tolist() == [1.0, -4.0, 0.5 - 0.5 - 0.5, 0.5, 4.0]
    # a chain: row 1 has the tokens of rows 0 and 1 behind it; a tree: row 2 not row 1's
    out, _ = oq.adjust(x, [0, 3], tok=[3, 4, 3], frequency=[1.0])
    assert out[:, 3].tolist() == [-0.5, -0.5, -1.5] and out[:, 4].tolist() == [4.0, 3.0, 3.0]
    out, _ = oq.adjust(x, [0, 3], tok=[3, 4, 3], frequency=[1.0], mask=np.array([[1], [3], [5]]))
    assert out[:, 4].tolist() == [4.0, 3.0, 4.0]
    # a bias comes before the penalties, the later entry counts; what is not allowed is -inf
    out, _ = oq.adjust(x, [0, 1], history=[[0]], repetition=[2.0], bias=[[(0, 9.0), (0, -6.0)]],
                       allowed=np.array([[0b01111]] * 3))
    assert out[0].tolist() == [-8.0, -2.0, 1.0, 0.5, -np.inf]
