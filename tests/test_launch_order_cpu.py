"""Kernels that may start before the one before them on the stream has ended (programmatic
dependent launches) wait for it before they write to memory: what they write may lie where
the kernel before still reads.  Read from the sources, since a missing wait shows on a GPU
only now and then."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_310_gb300", "csrc")
WAIT = "grid_dependency_wait();"
# through a pointer of the arguments, or a helper that stores; the error flag is the library's own
WRITES = [r"\*\s*p\.\w+\s*[+|]?=[^=]", r"\bp\.\w+\[[^;]*\]\s*[+|]?=[^=]", r"\bstore_\w+(<[^>]*>)?\(", r"atomic\w+\(\s*&?p\.",
          r"\bst\.global", r"\bred\.global", r"\*reinterpret_cast<[^;]*>\(p\.[^;]*\)\s*="]


def kernels():
    """name -> body, without comments, of every kernel in the sources."""
    found = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__[^;{]*?\b(?!__launch_bounds__)(\w+)\s*\((?=[^;{]*\{)", text):
            at = text.index("{", m.end())
            depth, end = 0, at
            while True:
                depth += (text[end] == "{") - (text[end] == "}")
                end += 1
                if depth == 0:
                    break
            found[m.group(1)] = text[at:end]
    return found


def launched_early():
    names = set()
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        text = open(path).read()
        names |= set(re.findall(r"launch_dependent\(\s*(\w+)", text)) | set(re.findall(r"cudaLaunchKernelEx\(&cfg,\s*(\w+)", text))
    return names


def test_the_kernels_are_found():
    assert {"work_list_kernel", "kv4_append_kernel", "scores_kernel", "select_kernel", "merge_kernel"} <= launched_early()
    assert launched_early() <= set(kernels())


def test_a_write_is_recognised():
    for text in ("*p.work_next = 0;", "p.work_list[pos + g] = x;", "store_out<T>(p.out, i, 0.f, f);", "atomicAdd(p.n, 1);"):
        assert any(re.search(w, text) for w in WRITES)
    for text in ("const int L = p.context_lens[s];", "if (p.a[i] == 0) x = 1;", "hist[i] = 0;", "set_error(p.err, kErrLength);"):
        assert not any(re.search(w, text) for w in WRITES)


@pytest.mark.parametrize("name", sorted(launched_early()))
def test_nothing_is_written_before_the_wait(name):
    body = kernels()[name]
    assert WAIT in body
    before = body[:body.index(WAIT)]
    for w in WRITES:
        assert not re.search(w, before), re.search(w, before).group(0)
