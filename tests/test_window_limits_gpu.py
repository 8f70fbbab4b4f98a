"""Windows and sinks past what 32 bits hold compute attention over every token."""
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
from window_model import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(2 ** 31, 0), (2 ** 32 + 5, 3), (1 << 40, 2 ** 32), (3, 2 ** 32), (1, 1 << 40)])
def test_decode(window, sinks, dtype):
    c = Case(316_000, [700, 33, 0], 700, 700, 8, 2, 64, 16, dtype).cuda()
    out = torch.empty_like(c.g_q)
    pkv.paged_attention_decode_window(c.g_q, c.g_k, c.g_v, c.g_tables, c.g_lens, c.scale, out, window=window, sinks=sinks,
                                      max_context_len=700)
    c.check(out)
    assert pkv.device_error() == 0


@pytest.mark.parametrize("window,sinks", [(2 ** 32 + 5, 3), (3, 2 ** 32)])
def test_prefill(window, sinks):
    c = Case(316_010, [700, 33], 700, 700, 8, 2, 64, 16, "f16", new=[300, 4]).cuda()
    out = torch.empty_like(c.g_q)
    pkv.paged_attention_prefill_window(c.g_q, c.g_k, c.g_v, c.g_tables, c.g_lens, c.g_start, c.scale, out, window=window,
                                       sinks=sinks, max_context_len=700)
    c.check(out)
    assert pkv.device_error() == 0
