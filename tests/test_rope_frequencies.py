"""Scaled rotary frequencies against their formulas, every pair of them, on the CPU.

ntk: base factor^(rot / (rot - 2)), so that pair i turns base^(-2 i / rot) factor^(-2 i / (rot - 2)).
yarn (Peng et al., 2023): with T turns over the original length, a pair keeps the part
g = (T - slow) / (fast - slow), held to 0..1, of its frequency and has the rest divided by the factor.
Both are formed here by logarithms, apart from a few roundings of float64 alike (rtol 1e-12: a power's
argument of up to log(base factor^2) = 20 is off by 20 * 2^-53 * 4 at most)."""
import math

import pytest

nf4 = pytest.importorskip("bit_quantized_fine_nf4_amd")


@pytest.mark.parametrize("rot", [2, 4, 8, 64, 96, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 2.0])
@pytest.mark.parametrize("factor", [1.0, 1.5, 8.0, 40.0])
def test_ntk(rot, base, factor):
    got, scale = nf4.qlora_rope_freqs(rot, base=base, scaling="ntk", factor=factor)
    assert scale == 1.0
    for i, f in enumerate(got.tolist()):
        slow = 2 * i / (rot - 2) * math.log(factor) if rot > 2 else 0.0
        assert f == pytest.approx(math.exp(-2 * i / rot * math.log(base) - slow), rel=1e-12)


@pytest.mark.parametrize("rot", [2, 8, 64, 96, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("factor,original,slow,fast", [(8.0, 2048, 1.0, 32.0), (4.0, 4096, 0.0, 10.0),
                                                       (40.0, 4096, 1.0, 32.0), (1.0, 1, 2.0, 3.5)])
def test_yarn(rot, base, factor, original, slow, fast):
    got, scale = nf4.qlora_rope_freqs(rot, base=base, scaling="yarn", factor=factor, original=original, slow=slow,
                                      fast=fast)
    assert scale == pytest.approx(1 + math.log(factor) / 10, rel=2.0 ** -23)
    between = 0
    for i, f in enumerate(got.tolist()):
        plain = math.exp(-2 * i / rot * math.log(base))
        turns = original * plain / math.tau
        if turns <= slow:
            want = plain / factor
        elif turns >= fast:
            want = plain
        else:
            between += 1
            want = plain * ((turns - slow) * factor + (fast - turns)) / ((fast - slow) * factor)
        assert f == pytest.approx(want, rel=1e-12)
    assert between or rot < 64 or original == 1
