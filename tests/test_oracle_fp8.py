"""The block-128 FP8 oracle against closed forms, torch's float8_e4m3fn and its own definition."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp8, mx


def test_scale_is_the_smallest_power_of_two_that_fits():
    for amax, e in ((448.0, 0), (np.nextafter(448.0, 1e9), 1), (447.0, 0), (224.0, -1), (224.1, 0), (1.0, -8), (1.75, -8),
                    (np.nextafter(1.75, 2), -7), (0.0, -126), (2.0 ** -130, -126), (448 * 2.0 ** -126, -126),
                    (449 * 2.0 ** -126, -125), (3.4e38, 120)):
        assert fp8.scale_of(amax) == 2.0 ** e, amax
    rng = np.random.default_rng(1)
    amax = np.exp(rng.uniform(-60, 60, 4000))
    s = fp8.scale_of(amax)
    assert np.all(amax / s <= 448) and np.all(amax / (s / 2) > 448)


def test_codes_are_nearest_with_ties_to_even():
    # 448 pins the scale to 1; 17 lies between 16 and 18 (codes 0x58, 0x59), 19 between 18 and 20
    v = np.zeros((1, 128))
    v[0, :8] = [448, 17, 19, -17, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -11, 0.0]
    codes, s = fp8.quantize(v)
    assert s[0, 0] == 1.0
    assert codes[0, :8].tolist() == [0x7E, 0x58, 0x5A, 0xD8, 0x00, 0x02, 0x80, 0x00]


@pytest.mark.parametrize("block_rows", [1, 128])
def test_against_torch_float8(block_rows):
    rng = np.random.default_rng(2)
    v = (rng.standard_normal((150, 272)) * np.exp(rng.uniform(-6, 6, (150, 1)))).astype(np.float32).astype(np.float64)
    codes, s = fp8.quantize(v, block_rows)
    assert s.shape == (150 if block_rows == 1 else 2, 3)
    q = torch.from_numpy((v / fp8.spread(s, block_rows, 150, 272)).astype(np.float32)).to(torch.float8_e4m3fn)
    assert np.array_equal(q.view(torch.uint8).numpy(), codes)
    assert np.array_equal(q.double().numpy(), mx.e4m3_to_f64(codes))
    err = np.abs(fp8.to_f64(codes, s, block_rows) - v)
    S = fp8.spread(s, block_rows, 150, 272)
    assert np.all(err <= np.maximum(np.abs(v) * 2.0 ** -4, S * 2.0 ** -10))  # half a step, or half the smallest subnormal


def test_bad_blocks_are_nan_and_alone():
    v = np.ones((3, 256))
    v[1, 5], v[2, 200] = np.nan, -np.inf
    codes, s = fp8.quantize(v)
    assert np.isnan(s[1, 0]) and np.isnan(s[2, 1]) and np.isfinite(s).sum() == 4
    assert np.all(codes[1, :128] == 0) and np.all(codes[2, 128:] == 0) and np.all(codes[0] == codes[1, 200])
    assert np.isnan(fp8.quantize(v, 128)[1]).tolist() == [[True, True]]


def test_expert_equals_a_composition_in_torch():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 160))
    w = [fp8.to_f64(*fp8.quantize(rng.standard_normal(s) * 0.1, 128), 128) for s in ((96, 160), (96, 160), (160, 96))]

    def q(t):
        t = t.numpy()
        pad = np.zeros((t.shape[0], -(-t.shape[1] // 128) * 128))
        pad[:, :t.shape[1]] = t
        m = np.abs(pad.reshape(t.shape[0], -1, 128)).max(2)
        s = np.repeat(2.0 ** np.ceil(np.log2(m / 448)), 128, 1)[:, :t.shape[1]]
        return torch.from_numpy((t / s).astype(np.float32)).to(torch.float8_e4m3fn).double() * torch.from_numpy(s)

    xq = q(torch.from_numpy(x))
    h = torch.nn.functional.silu(xq @ torch.from_numpy(w[0]).T) * (xq @ torch.from_numpy(w[1]).T)
    y = q(h) @ torch.from_numpy(w[2]).T
    np.testing.assert_allclose(fp8.swiglu_expert(x, *w), y.numpy(), rtol=1e-12, atol=1e-12)
