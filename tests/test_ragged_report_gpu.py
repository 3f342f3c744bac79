"""Lengths and prefix sums out of range are reported wherever in the batch they are."""

import numpy as np
import pytest
import torch

from gqa_attention_split_gb300 import api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    api.lib()


def _reported(call):
    call()
    with pytest.raises(api.GqaError) as e:
        api.check()
    assert e.value.code == api.GQA_ERR_DEVICE_BAD_INPUT


# a cache of 512 slots or less is not cut, a larger one is
@pytest.mark.parametrize("S_max", [64, 1024])
@pytest.mark.parametrize("row", [0, 31, 32, 70, 99])
@pytest.mark.parametrize("what", ["context", "drafts"])
def test_tree_reports_bad_rows_anywhere(S_max, row, what):
    B, H_q, H_kv, d = 100, 4, 1, 64
    ctx, drafts = np.full(B, 9, np.int32), np.full(B, 2)
    if what == "context":
        ctx[row] = S_max + 1
    else:
        drafts[row] = 4
    n = int(drafts.sum())
    cu = torch.tensor([0] + list(np.cumsum(drafts)), dtype=torch.int32, device="cuda")
    x = [torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
         for s in ((n, H_q, d), (n, H_kv, d), (B, H_kv, S_max, d))]
    _reported(lambda: api.decode_tree(x[0], x[1], x[1], x[2], x[2], torch.from_numpy(ctx).cuda(),
                                      cu_seqlens=cu, max_tokens=3))
    ctx[row], good = 9, torch.arange(B + 1, dtype=torch.int32, device="cuda")  # and not without one
    api.decode_tree(x[0], x[1], x[1], x[2], x[2], torch.from_numpy(ctx).cuda(), cu_seqlens=good,
                    max_tokens=3)
    api.check()


# Prefix sums that go up and down: every other row holds all tokens. With the valid ones no launch has
# more blocks of queries than the tokens and rows allow; here it would be B / 2 times as many, past 32
# bits in the last case. Reported, nothing computed, and the next call is as ever.
@pytest.mark.parametrize("B,n,H_q", [(600, 500, 4), (2000, 500, 4), (65535, 300000, 128)])
def test_packed_rows_that_overlap_are_reported_and_not_computed(B, n, H_q):
    q = torch.empty(n, H_q, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(n, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[:500] = 0
    out, lse = torch.empty_like(q), torch.full((n, H_q), 9.0, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = n
    _reported(lambda: api.prefill_packed(q, k, k, cu, out=out, lse=lse))
    assert (lse == 9).all()
    cu = torch.full((B + 1,), 500, dtype=torch.int32, device="cuda")
    cu[0] = 0
    api.prefill_packed(q, k, k, cu, out=out, lse=lse)
    api.check()
    want = torch.log(torch.arange(1, 501, device="cuda"))[:, None].expand(-1, H_q)
    assert (lse[:500] - want).abs().max() < 1e-5 and (lse[500:] == 9).all()
