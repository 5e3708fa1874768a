"""The e4m3 oracle against torch's own conversion, and its block rule on small examples."""
import numpy as np
import pytest
import torch

from oracle import fp8


def test_every_code_and_every_midpoint():
    codes = np.arange(256, dtype=np.uint8)
    v = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp8.decode(codes)[~np.isnan(v)], v[~np.isnan(v)])
    assert np.array_equal(np.isnan(v), np.isnan(fp8.decode(codes)))
    t = fp8.TABLE
    mid = (t[1:] + t[:-1]) / 2
    q = np.concatenate([t, mid, np.nextafter(mid.astype(np.float32), np.float32(0)), -t, -mid,
                        np.nextafter(mid.astype(np.float32), np.float32(1e9))]).astype(np.float32)
    got = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.encode(q), got)


@pytest.mark.parametrize("rows", [1, 128])
def test_blocks(rows):
    x = np.zeros((130, 300), np.float32)
    x[0, 0], x[0, 129], x[129, 299] = 448.0, -2.0, 1.0
    codes, scales = fp8.pack(x, rows)
    assert codes.shape == x.shape and scales.shape == (-(-130 // rows), 3)
    assert scales[0, 0] == 1.0 and scales[0, 2] == 1.0  # the largest value 448, and an empty block
    assert scales[0, 1] == np.float32(2) / np.float32(448)
    back = fp8.dequant(codes, scales, rows)
    assert np.allclose(back, x, rtol=2.0 ** -22)


def test_sort():
    ids = np.array([[1, 0], [-1, 1], [0, 7], [1, 1]])
    tokens, pos, offsets = fp8.sort(ids, 3)
    assert tokens.tolist() == [0, 2, 0, 1, 3, 3, -1, -1]
    assert pos.tolist() == [[2, 0], [-1, 3], [1, -1], [4, 5]]
    assert offsets.tolist() == [0, 2, 6, 6]
