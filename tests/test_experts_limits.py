"""The limits of the expert operators' C ABI on the host, no device needed."""
import pytest

from differentiable_exact_budget_amd import experts

INVALID = 1
FAKE = 4096  # a non-NULL, 16-byte aligned address that is never dereferenced
WIDEST = 0x7FFF0000


@pytest.mark.parametrize("width", [WIDEST + 1, 2 ** 31 - 31, 2 ** 31 - 15, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_products_refuse_widths_whose_tiles_end_past_2_to_the_31(dtype, width):
    """A sum of nearly 2^31 terms, or so many columns, counted in steps and
    tiles from there, would pass 32 bits: shares of the sum came out empty."""
    lib = experts.lib()
    for size in ((width, 8), (8, width)):
        assert lib.lapsum_expert_linear(FAKE, FAKE, None, dtype, 1, *size, 1, FAKE, 0, FAKE, None, None) == INVALID
        assert lib.lapsum_expert_linear_vjp(FAKE, FAKE, None, FAKE, dtype, 1, *size, 1, FAKE, 0, FAKE, FAKE, FAKE, FAKE,
                                            None) == INVALID
        assert lib.lapsum_expert_linear_vjp_scratch_bytes(dtype, 1, *size, 1, 2, 1) == 0
    assert lib.lapsum_expert_linear_vjp_scratch_bytes(dtype, 1, 8, WIDEST, 1, 2, 1) > 0
