"""Pins of the 64-bit model of the 8-bit K/V cache (CPU): hand-derived codes, rotation, masks,
lists."""
import numpy as np
import torch

from oracle import kv8 as model


def test_e4m3_grid_matches_torch():
    want = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(model.e4m3_values()[:127], want)
    vals = np.concatenate([want, -want[1:]])
    back = torch.from_numpy(vals).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(model.code_bytes(vals, "e4m3"), back)


def test_nearest_codes():
    y = [0.5, 1.5, -0.5, -2.5, 126.5, 127.4, 500.0, np.nan, np.inf, -np.inf, 0.49999999]
    assert model.nearest(y, "int8").tolist() == [0, 2, 0, -2, 126, 127, 127, 0, 127, -127, 0]
    # 17 lies between 16 and 18, 19 between 18 and 20: the even mantissas are 16 and 20
    y = [17.0, 19.0, 17.0000001, 2.0 ** -10, 3 * 2.0 ** -10, 464.0, 1e9, -17.0]
    want = [16.0, 20.0, 18.0, 0.0, 2.0 ** -8, 448.0, 448.0, -16.0]
    assert model.nearest(y, "e4m3").tolist() == want


def test_rotation_by_a_quarter_turn():
    x = np.arange(1.0, 9.0)[None]
    c, s = np.zeros(2), np.ones(2)
    assert model.rotate(x, c, s, True).tolist() == [[-2, 1, -4, 3, 5, 6, 7, 8]]
    assert model.rotate(x, c, s, False).tolist() == [[-3, -4, 1, 2, 5, 6, 7, 8]]


def test_append_recodes_older_tokens_when_the_scale_grows():
    p = model.Pool(2, 1, 8, 4, "int8")
    x = np.zeros((1, 1, 8))
    x[0, 0, :2] = [127.0, 3.0]
    p.append(x, x, [1], 0)
    assert p.ks[1, 0] == 1.0 and p.k[1, 0, 0, 1] == 3.0
    y = np.zeros((1, 1, 8))
    y[0, 0, 2] = -254.0
    p.append(y, y, [1], 1)
    # scale 2: 127 / 2 = 63.5 and 3 / 2 = 1.5 are ties and go to the even codes
    assert p.ks[1, 0] == 2.0
    assert p.k[1, 0, 0, :2].tolist() == [64.0, 2.0] and p.k[1, 0, 1, 2] == -127.0
    assert p.km[1, 0, :3].tolist() == [64.0, 2.0, -127.0]
    assert not p.ks[0].any()


def test_attention_of_equal_keys_is_the_mean_and_empty_rows_are_zero():
    p = model.Pool(1, 1, 8, 4, "int8")
    k, v = np.ones((3, 1, 8)), np.zeros((3, 1, 8))
    v[:, 0, 0] = [127.0, 1.0, -127.0]
    p.append(k, v, [0], 0)
    q = np.ones((5, 1, 8))
    out, lse, size, _ = p.attend(q, [0], 3, True, 0.5)
    # 5 queries over 3 keys: the first two see nothing
    assert not out[:2].any() and np.isneginf(lse[:2]).all()
    assert np.allclose(out[2:, 0, 0], [127.0, 64.0, 1 / 3]) and np.allclose(lse[4], 4 + np.log(3))
    assert np.allclose(size[4, 0, 0], 255 / 3)


def test_selection_keeps_ends_and_prefers_low_indices():
    p = model.Pool(5, 1, 8, 4, "int8")
    for page, m in enumerate([0.0, 2.0, 2.0, 5.0, 1.0]):
        p.km[page, 0, 0] = m
    q = np.zeros((1, 1, 8))
    q[0, 0, 0] = 1.0
    table = [0, 1, 2, 3, 4]
    assert p.select(q, table, 20, False, 1, 2, 0, 0)[0, 0].tolist() == [1, 3]
    assert p.select(q, table, 20, False, 1, 3, 1, 1)[0, 0].tolist() == [0, 3, 4]
    assert p.select(q, table, 9, False, 1, 4, 0, 0)[0, 0].tolist() == [0, 1, 2, -1]
    assert p.select(q, [0, 7, 2, 3, 4], 20, False, 1, 2, 0, 0)[0, 0].tolist() == [2, 3]
