"""Pins of oracle/latent.py: closed forms, exact rationals and torch's float64 routines."""

from fractions import Fraction

import numpy as np
import torch

from oracle import latent


def test_rmsnorm_closed_form_and_torch():
    # mean square of (3, 4, 0, 0) is 25/4: the norm divides by 2.5
    y = latent.rmsnorm_ref(np.array([[3.0, 4.0, 0.0, 0.0]]), np.array([1.0, 2.0, 1.0, 1.0]), 0.0)
    np.testing.assert_array_equal(y, [[1.2, 3.2, 0.0, 0.0]])
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((5, 48)), rng.standard_normal(48)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (48,), torch.from_numpy(w), 1e-6).numpy()
    np.testing.assert_allclose(latent.rmsnorm_ref(x, w, 1e-6), want, rtol=1e-14)


def test_token_code_is_the_least_power_of_two():
    rng = np.random.default_rng(1)
    y = rng.standard_normal((200, 8)) * np.exp2(rng.integers(-30, 30, (200, 1)))
    y[0] = 448.0          # scale exactly 1
    y[1] = 448.0 * 2 ** 7
    y[2] = 0.0            # the floor: 1e-10 / 448 -> 2^-42
    y[3] = np.nextafter(448.0, 500.0)
    codes = latent.token_code_ref(y)
    assert codes[0] == 127 and codes[1] == 134 and codes[2] == 127 - 42 and codes[3] == 128
    for row, c in zip(y, codes):
        s = Fraction(max(float(np.abs(row).max()), 1e-10)) / 448
        assert Fraction(2) ** int(c - 127) >= s > Fraction(2) ** int(c - 128)
    assert latent.token_code_ref(np.array([[1.0, np.nan], [np.inf, 0.0], [1e30, 0.0]])).tolist() == [255, 255, 167]


def test_e8m0_values_are_torchs():
    codes = np.arange(255, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e8m0fnu).float().double().numpy()
    np.testing.assert_array_equal(latent.e8m0_value(codes), want)
    assert np.isnan(latent.e8m0_value(np.array([255])))[0]


def test_attention_against_torch_and_empty_rows():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((6, 16)), rng.standard_normal((9, 16)), rng.standard_normal((9, 4))
    sees = np.array([0, 1, 5, 9, -3, 8])
    o, mag, reach = latent.attention_ref(q, k, v, sees, 0.3)
    mask = torch.arange(9)[None, :] < torch.from_numpy(sees)[:, None]
    s = (torch.from_numpy(q @ k.T) * 0.3).masked_fill(~mask, float("-inf"))
    want = torch.softmax(s, dim=-1) @ torch.from_numpy(v)
    live = sees > 0
    np.testing.assert_allclose(o[live], want.numpy()[live], rtol=1e-12, atol=1e-14)
    assert (o[~live] == 0).all() and (mag >= np.abs(o) - 1e-15).all()
    np.testing.assert_array_equal(o[1], v[0])  # one key: its value
    assert reach[3] >= np.abs(0.3 * (k @ q[3])).max()
