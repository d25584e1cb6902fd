"""The fp64 reference of the block-scaled e4m3 operators against hand values, torch's conversions and differences."""
import numpy as np
import pytest
import torch

from oracle import e4m3_to_f64, fp8


def test_codes_match_the_type_conversion():
    v = torch.randn(4096, generator=torch.Generator().manual_seed(1)) * 60
    v = torch.cat([v.clamp(-448, 448), torch.tensor([0.0, -0.0, 448, -448, 2**-9, 2**-10, 3 * 2**-10, 17.0, 19.0, 2**-7])])
    assert np.array_equal(fp8.e4m3_codes(v.double().numpy()), v.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("amax,byte", [(448.0, 127), (450.0, 128), (224.0, 126), (1.0, 127 - 8), (1.75, 127 - 8),
                                       (1.76, 127 - 7), (0.0, 127), (2.0**-133, 3), (448 * 2.0**-124, 3),
                                       (449 * 2.0**-124, 4), (3.3e38, 247), (np.inf, 255), (np.nan, 255)])
def test_scales(amax, byte):
    x = np.zeros((1, 128))
    x[0, 77] = -amax
    codes, scales = fp8.quantize(x)
    assert scales[0, 0] == byte
    if byte < 255:
        v = fp8.values(codes, scales)
        assert abs(v[0, 77] + amax) <= 2.0**-4 * amax and not v[0, :77].any()
    else:
        assert np.isnan(fp8.values(codes, scales)).all()


def test_blocks_end_short():
    x = np.ones((130, 144))
    x[128:, :128] = 2.0**20
    codes, scales = fp8.quantize(x, 128)
    assert scales.shape == (2, 2) and scales[1, 0] == 127 + 20 - 8 and scales[1, 1] == 127 - 8
    assert np.array_equal(fp8.values(codes, scales, 128), x)
    assert e4m3_to_f64(codes).max() == 256


def test_gradients_by_differences():
    rng = np.random.default_rng(3)
    h, w, dy = rng.standard_normal((3, 24)), rng.standard_normal(24), rng.standard_normal((3, 24))
    g = fp8.rms_norm_backward(h, w, dy, None, 1e-3)
    f = lambda h, w: (fp8.rms_norm(h, w, 1e-3) * dy).sum()
    t = 1e-6
    for at in ((0, 0), (1, 7), (2, 23)):
        e = np.zeros_like(h)
        e[at] = t
        assert abs((f(h + e, w) - f(h - e, w)) / (2 * t) - g["x"][0][at]) < 1e-7
    for c in (0, 11):
        e = np.zeros_like(w)
        e[c] = t
        assert abs((f(h, w + e) - f(h, w - e)) / (2 * t) - g["weight"][0][c]) < 1e-7
    x, v = rng.standard_normal((4, 16)), rng.standard_normal((8, 16))
    dy = fp8.values(*fp8.quantize(rng.standard_normal((4, 8))))   # already what its quantisation stands for
    g = fp8.linear_backward(x, v, dy)
    f = lambda x, v: (fp8.linear(x, v)[0] * dy).sum()
    e = np.zeros_like(x)
    e[2, 5] = t
    assert abs((f(x + e, v) - f(x - e, v)) / (2 * t) - g["x"][0][2, 5]) < 1e-7
    e = np.zeros_like(v)
    e[7, 3] = t
    assert abs((f(x, v + e) - f(x, v - e)) / (2 * t) - g["weight"][0][7, 3]) < 1e-7
