"""Nothing that the kernel before may have written is relied on before the wait for it: a kernel that
starts early reads no memory of the call there, but for the decode work list's lengths, which it
reads again after the wait.  Read from the sources."""
import re

import pytest

from test_launch_order_cpu import WAIT, kernels, launched_early

# through a pointer of the arguments
READS = [r"\bp\.\w+\[", r"\*\s*p\.\w+", r"__ld\w+\(", r"\bld\.global"]


def before(name):
    body = kernels()[name]
    return body[:body.index(WAIT)]


def test_a_read_is_recognised():
    for text in ("const int L = p.context_lens[s];", "x = *p.work_count;", "y = __ldcg(p.context_lens + s);"):
        assert any(re.search(r, text) for r in READS), text
    for text in ("const int H = p.num_kv_heads / p.heads;", "hist[i] = 0;"):
        assert not any(re.search(r, text) for r in READS), text


@pytest.mark.parametrize("name", sorted(launched_early() - {"work_list_kernel"}))
def test_nothing_is_read_before_the_wait(name):
    for r in READS:
        assert not re.search(r, before(name)), re.search(r, before(name)).group(0)


def test_lengths_read_early_are_read_again():
    body = kernels()["work_list_kernel"]
    early, after = before("work_list_kernel"), body[body.index(WAIT) + len(WAIT):]
    # one length a thread, past the SM's L1, and nothing flagged
    assert len(re.findall(r"p\.context_lens", early)) == 1 and "__ldcg(p.context_lens + threadIdx.x)" in early
    assert "set_error" not in early
    # held against what the wait made visible, and not looked at again
    assert re.match(r"\s*const int held = mine \? p\.context_lens\[threadIdx\.x\] : 0;\s*"
                    r"if \(__syncthreads_or\(!guess \|\| held != guessed\)\) \{", after)
    assert after.count("guessed") == 1
