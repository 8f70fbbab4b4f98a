"""Tokens of a padded batch: a negative position makes a token padding whatever its slot is."""
import torch

import pytest

import paged_kv_cache_310_gb300 as pkv
from test_rotary_gpu import Case, append, pools

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [6, 700])
def test_the_slot_of_a_padding_token_does_not_matter(tokens):
    c = Case(316_600, tokens, 4, 2, 64, "bf16", 64, norm="q")
    kc, vc = pools(c, tokens // 4, 8, 2)
    was = [kc.clone(), vc.clone()]
    slots = torch.arange(tokens)
    c.positions[1::3] = -1
    slots[1::3] = torch.tensor([tokens * 100, 1 << 40, (1 << 63) - 1, -5, 0]).repeat(tokens)[:len(slots[1::3])]
    live = c.positions >= 0
    out = append(c, slots, kc, vc)
    assert pkv.device_error() == 0
    assert (out[~live.cuda()] == 7).all() and not (out[live.cuda()] == 7).all(-1).any()
    rows = lambda x: x.transpose(1, 2).reshape(-1, 2, 64)
    mine = slots[live].cuda()
    assert torch.equal(rows(vc)[mine], c.v[live.cuda()])
    rest = torch.ones(len(rows(vc)), dtype=torch.bool, device="cuda")
    rest[mine] = False
    assert all(torch.equal(rows(a)[rest], rows(b)[rest]) for a, b in zip((kc, vc), was))


def test_a_slot_out_of_range_of_a_token_that_counts_is_flagged():
    c = Case(316_610, 3, 4, 2, 64, "bf16", 64)
    kc, vc = pools(c, 4, 8, 2)
    c.positions[0], c.positions[1] = -1, 0
    append(c, torch.tensor([99, 32, 3]), kc, vc)
    assert pkv.device_error() == 5 and (c.q_out[:2] == 7).all() and not (c.q_out[2] == 7).any()
