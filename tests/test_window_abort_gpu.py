"""The windowed prefill's tensor-core kernel gives up part-way when its pipeline waits are bounded far
below what they take, returns with the timeout status, and leaves the context usable; the kernels for
few rows have no such waits and do not mind the bound."""
import time

import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
from test_window_prefill_gpu import kernel_of, run
from window_model import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,group,hkv,lens,new,window,kernel", [
    (128, 8, 2, [2000], [1000], 600, "shared"), (64, 4, 4, [2500], [1100], 700, "shared"),
    (128, 8, 2, [4100], [4000], 64, "pairs"), (64, 16, 4, [1200, 700], [1000, 650], 129, "pairs")])
def test_prefill_gives_up_and_the_context_survives(d, group, hkv, lens, new, window, kernel):
    c = Case(314_400, lens, window, 4, group * hkv, hkv, d, 16, "bf16", new=new)
    assert kernel_of(c) == kernel and pkv.device_error() == 0
    pkv.set_wait_limit(1_000)
    try:
        t0 = time.perf_counter()
        run(c)
        status = pkv.device_error()
        elapsed = time.perf_counter() - t0
    finally:
        pkv.set_wait_limit(0)
    assert status == 6 and elapsed < 10.0 and pkv.device_error() == 0
    c.check(run(c))
    assert pkv.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_rows_do_not_wait(dtype):
    c = Case(314_410, [900, 40], 300, 4, 8, 2, 64, 16, dtype).cuda()
    out = torch.empty_like(c.g_q)
    pkv.set_wait_limit(1_000)
    try:
        pkv.paged_attention_decode_window(c.g_q, c.g_k, c.g_v, c.g_tables, c.g_lens, c.scale, out, window=300, sinks=4,
                                          max_context_len=900)
        assert pkv.device_error() == 0
    finally:
        pkv.set_wait_limit(0)
    c.check(out)
