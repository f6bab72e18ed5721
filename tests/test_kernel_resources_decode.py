"""Registers of a decoding step's kernels: none of them keeps registers in memory.
Runs without a GPU."""
import pytest

from test_kernel_resources import kernels  # noqa: F401

NAMES = ("w4a16_few_kernel", "w4a16_many_kernel", "w4a16_join_kernel", "cache_write_kernel", "cache_read_kernel",
         "attention_tokens_kernel", "attention_rows_kernel", "attention_both_kernel", "attention_join")


@pytest.mark.parametrize("name", NAMES)
def test_no_scratch(kernels, name):  # noqa: F811
    mine = {k: v for k, v in kernels.items() if name in k}
    assert mine
    for k, v in mine.items():
        assert v[".private_segment_fixed_size"] == 0 and v[".vgpr_spill_count"] == 0, (
            k, v[".private_segment_fixed_size"], v[".vgpr_spill_count"])
