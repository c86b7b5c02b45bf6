"""What fixes the 4-bit cache's oracle other than itself: hand-worked rows, torch's
own e4m3 cast, and the grids' spacing."""

import numpy as np
import torch

from oracle import kv4


def test_grids():
    bits = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv4.E4M3, bits)
    # sign, exponent (bias 1), one mantissa bit
    assert kv4.CODES.tolist() == [m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1) for e in range(4) for m in range(2)]


def test_nearest_is_torchs_e4m3_cast():
    g = torch.Generator().manual_seed(1)
    x = torch.rand(20000, generator=g) * 2.0 ** torch.randint(-12, 9, (20000,), generator=g)
    mids = torch.tensor((kv4.E4M3[1:] + kv4.E4M3[:-1]) / 2).float()
    x = torch.cat([x.clamp(max=448), mids, torch.zeros(1)])
    assert np.array_equal(kv4.nearest(x.double().numpy(), kv4.E4M3), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_a_row_by_hand():
    x = np.zeros(32)
    # largest magnitude 12: scale 2, codes x / 2; 0.5, 1.5, 2.5, 3.5, 5 and 7 stand on borders
    x[:16] = [12, -12, 0.5, 1.5, 2.5, 3.5, 5, 7, 10, -0.5, 1, 2, 3, 4, 6, 8]
    codes, sf = kv4.quantise(x)
    assert kv4.E4M3[sf].tolist() == [2, 0]
    want = [12, -12, 0, 2, 2, 4, 4, 8, 8, 0, 1, 2, 3, 4, 6, 8]
    assert kv4.values(codes, sf)[:16].tolist() == want and not kv4.values(codes, sf)[16:].any()
    assert codes[0] == 7 | 15 << 4                             # the even value in the low half
    codes, sf = kv4.quantise(x * 2.0 ** -20, 2.0 ** -20)       # the factor moves the range
    assert kv4.values(codes, sf, 2.0 ** -20)[:16].tolist() == [w * 2.0 ** -20 for w in want]


def test_scale_to_nearest_and_the_ends_of_its_range():
    # 6.375 / 6 = 1.0625 lies between 1 and 1.125: ties to the even mantissa; the value is cut to 6
    codes, sf = kv4.quantise(np.full(16, 6.375))
    assert kv4.E4M3[sf] == [1.0] and (kv4.values(codes, sf) == 6).all()
    codes, sf = kv4.quantise(np.array([np.inf, -np.inf, 1e30, 2688.0] + [1.0] * 12))
    assert kv4.values(codes, sf)[:4].tolist() == [2688, -2688, 2688, 2688]
    codes, sf = kv4.quantise(np.full(16, 6 * 2.0 ** -10))      # half the smallest scale: to 0
    assert sf == [0] and not kv4.values(codes, sf).any()
    codes, sf = kv4.quantise(np.array([np.nan] + [1.0] * 15))
    assert sf == [127] and np.isnan(kv4.values(codes, sf)).all()


def test_error_is_half_a_step():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(200, 128)) * 2.0 ** rng.integers(-3, 4, size=(200, 1))
    codes, sf = kv4.quantise(x)
    scale = np.repeat(kv4.E4M3[sf], 16, axis=-1)
    off = np.abs(kv4.values(codes, sf) - x)
    m = np.abs(x) / scale
    step = np.where(m <= 2, 0.5, np.where(m <= 4, 1.0, 2.0))
    # beyond 6 the scale itself was rounded down, by at most a sixteenth
    assert (off <= np.where(m <= 6, step / 2, 6 / 16 + 1e-12) * scale + 1e-15).all()
