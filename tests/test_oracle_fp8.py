"""The 64-bit forms of the 8-bit operators against independent statements of the same: the
e4m3 codec against every code and every midpoint, scales against their definition, the norm's
gradients against differences (CPU)."""
import numpy as np
import pytest

from oracle import fp8


def test_e4m3_codes_and_rounding():
    v = fp8.e4m3_decode(np.arange(256))
    pos = v[:127]
    assert np.all(np.diff(pos) > 0) and pos[-1] == 448.0 and pos[1] == 2.0 ** -9
    assert np.isnan(v[127]) and np.isnan(v[255])
    assert np.array_equal(v[128:255], -pos)
    assert np.array_equal(fp8.e4m3_round(pos), pos)
    mid = (pos[:-1] + pos[1:]) / 2
    even = np.where(np.arange(126) % 2 == 0, pos[:-1], pos[1:])  # the code with a zero last bit
    assert np.array_equal(fp8.e4m3_round(mid), even)
    assert np.array_equal(fp8.e4m3_round(-mid), -even)
    assert np.array_equal(fp8.e4m3_round(mid * (1 + 2.0 ** -40)), pos[1:])
    assert np.array_equal(fp8.e4m3_round(mid * (1 - 2.0 ** -40)), pos[:-1])


def test_e4m3_codes_match_torch():
    import torch
    code = torch.arange(256, dtype=torch.uint8)
    t = code.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, fp8.e4m3_decode(code.numpy()), equal_nan=True)


def test_scales():
    for k in (-126, -3, 0, 40):
        s = 2.0 ** k
        assert fp8.scale_of(np.array(448 * s)) == s
        assert fp8.scale_of(np.array(448 * s * (1 + 2.0 ** -20))) == 2 * s
    assert fp8.scale_of(np.array(0.0)) == 2.0 ** -126
    v = np.full((1, 130), np.inf)
    v[0, 5], v[0, 129] = -3.0, np.nan
    assert np.array_equal(fp8.block_max(v), [[3.0, 0.0]])


@pytest.mark.parametrize("N,H,res", [(3, 40, True), (1, 8, False)])
def test_rmsnorm_gradient_against_differences(N, H, res):
    rng = np.random.default_rng(N + H)
    r, w, dy = rng.standard_normal((N, H)), rng.standard_normal(H), rng.standard_normal((N, H))
    dres = rng.standard_normal((N, H)) if res else None
    f = lambda r_, w_: (fp8.rmsnorm(r_, w_, 1e-6)[0] * dy).sum() + (0 if dres is None else (dres * r_).sum())
    dx, dw, _, _ = fp8.rmsnorm_backward(dy, r, w, fp8.rmsnorm(r, w, 1e-6)[1], dres)
    h = 1e-6
    for _ in range(20):
        i, j = rng.integers(N), rng.integers(H)
        d = np.zeros((N, H)); d[i, j] = h
        assert (f(r + d, w) - f(r - d, w)) / (2 * h) == pytest.approx(dx[i, j], rel=1e-6, abs=1e-7)
        d = np.zeros(H); d[j] = h
        assert (f(r, w + d) - f(r, w - d)) / (2 * h) == pytest.approx(dw[j], rel=1e-6, abs=1e-7)


def test_grouped_is_a_dense_product_for_one_expert():
    rng = np.random.default_rng(0)
    a, w = rng.standard_normal((5, 32)), rng.standard_normal((1, 7, 32))
    one = np.ones((1, 1))
    out, _ = fp8.grouped(a, one, w, one[None], [0, 5], np.arange(5))
    assert np.allclose(out, a @ w[0].T, rtol=0, atol=0)
