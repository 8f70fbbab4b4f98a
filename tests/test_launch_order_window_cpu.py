"""A kernel that lets the next one start early has itself waited for the one before: the decode work
list reads context lengths before its own wait, and goes by that.  Read from the sources."""
import pytest

from test_launch_order_cpu import WAIT, kernels, launched_early

START = "grid_dependents_launch();"
# whose next kernel is one of the same call and reads nothing before its own wait, or that are ordinary launches
OTHERS = {"work_list_kernel", "append_kernel", "decode_simt_kernel"}


def test_these_kernels_are_looked_at():
    starts = {name for name, body in kernels().items() if START in body}
    assert {"rotary_kernel", "window_rows_kernel", "window_rows_f32_kernel", "window_prefill_kernel"} <= starts & launched_early()
    assert OTHERS <= starts and not {"append_kernel", "decode_simt_kernel"} & launched_early()


@pytest.mark.parametrize("name", sorted(n for n, body in kernels().items() if START in body and n not in OTHERS))
def test_the_wait_comes_first(name):
    body = kernels()[name]
    assert WAIT in body and body.index(WAIT) < body.index(START)
