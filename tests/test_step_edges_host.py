"""What of the serving-step operators' edges shows without a GPU."""

import pytest

import moe_expert_ffn_dispatch_gb300 as m
from moe_expert_ffn_dispatch_gb300 import layer


@pytest.fixture(scope="module")
def built():
    from moe_expert_ffn_dispatch_gb300 import _build
    _build.build()
    return m.lib()


@pytest.mark.parametrize("sizes", [(2 ** 32 + 100, 64, 64), (100, 2 ** 32 + 64, 64), (100, 64, 2 ** 32 + 64), (-2 ** 32 + 100, 64, 64),
                                   (100, 64, -2 ** 32 + 64), (2 ** 31, 64, 64)])
def test_w8_workspace_sizes_past_32_bits_are_not_cut(built, sizes):
    """ctypes would take each for the number that its low 32 bits are."""
    with pytest.raises(ValueError, match="32 bits"):
        layer._w8_workspace_bytes(*sizes, 0)


def test_w8_workspace_sizes_that_the_entry_refuses_still_reach_it(built):
    for sizes in ((-1, 64, 64), (100, 64, 40), (2 ** 31 - 1, 64, 64), (100, -2 ** 31 + 1, 64)):
        with pytest.raises(m.MoeError) as e:
            layer._w8_workspace_bytes(*sizes, 0)
        assert e.value.code == m.MOE_ERR_UNSUPPORTED_SHAPE
