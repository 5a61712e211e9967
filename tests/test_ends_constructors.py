"""What the norm of whole tokens refuses when it is made, before it looks for a GPU."""
import pytest

from long_convolution_sequence_rfft_amd import hyena


@pytest.mark.parametrize("kind", ["e5m2", "fp8", "", 8, [], True, False])
def test_formats(kind):
    with pytest.raises(ValueError, match="quantized must be"):
        hyena.ResidualNorm(1, 4, 64, quantized=kind)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("group", [0, 16, 48, 256, -32, "32"])
def test_groups(kind, group):
    with pytest.raises(ValueError, match="group must be"):
        hyena.ResidualNorm(1, 4, 768, quantized=kind, group=group)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_groups_without_eight_bits_or_a_fitting_width(group):
    with pytest.raises(ValueError, match="group must be"):
        hyena.ResidualNorm(1, 4, 768, group=group)
    with pytest.raises(ValueError, match="d must be a multiple of group"):
        hyena.ResidualNorm(1, 4, 5 * group + 16, quantized="int8", group=group)
