"""Frequencies of the rotation, on the host."""
import pytest
import torch


@pytest.mark.parametrize("dim,axes", [(2, 1), (3, 1), (4, 2), (6, 3), (7, 3)])
def test_the_base_cannot_scale_a_single_pair(dim, axes):
    # One pair's frequency is 1 whatever the base is: both the fastest, which stays, and the slowest, which is divided.
    import sparse_convolution_amd as igc
    with pytest.raises(ValueError, match="two pairs"):
        igc.rotary_frequencies(dim, axes=axes, scaling="base", factor=4.0)
    assert torch.equal(igc.rotary_frequencies(dim, axes=axes, scaling="base"), torch.ones(axes, 1))
    assert torch.equal(igc.rotary_frequencies(dim, axes=axes, scaling="linear", factor=4.0), torch.full((axes, 1), 0.25))


@pytest.mark.parametrize("dim,axes", [(4, 1), (8, 2), (64, 1), (64, 3)])
@pytest.mark.parametrize("factor", [0.5, 4.0])
def test_the_base_divides_the_slowest_and_leaves_the_fastest(dim, axes, factor):
    import sparse_convolution_amd as igc
    f, g = igc.rotary_frequencies(dim, axes=axes), igc.rotary_frequencies(dim, axes=axes, scaling="base", factor=factor)
    assert bool((g[:, 0] == 1).all())
    # Both are rounded to fp32 once: 2^-24 each, and powers in 64 bits.
    assert bool(((g[:, -1].double() * factor / f[:, -1].double() - 1).abs() < 2 * 2.0 ** -24 * (1 + 1e-6)).all())


@pytest.mark.parametrize("shape", [(0, 5), (0, 0)])
def test_frequencies_of_no_axis_are_refused(shape):
    # They would leave every channel as it is.
    from sparse_convolution_amd._selfattn import _turn
    with pytest.raises(ValueError, match="at least one axis"):
        _turn(torch.zeros(4, 0, dtype=torch.int32), torch.zeros(shape), 4, "half", 0)
