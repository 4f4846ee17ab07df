"""Failure detection of the backward without a GPU fault: with the test-only stall an
MMA issuer waits on a barrier that nobody signals; the items give up after their bound,
the error word reports it, and the next call on the same context is right."""
import pytest
import torch

import block_sparse_attention_tsr_gb300 as tsr
import workloads as W

pytestmark = pytest.mark.gpu

KEY_S, KEY_DP, QUERY_S, QUERY_DP = 1, 2, 4, 8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tsr.build()
    tsr.lib()


@pytest.mark.parametrize("where", [KEY_S, KEY_DP, QUERY_S, QUERY_DP, KEY_S | KEY_DP, 15])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,N", [(2, 700), (1, 2100)])       # the second: items in two parts
def test_bounded_wait_reports_timeout_and_context_survives(H, N, d, where):
    stall_and_recover(H, N, d, where)


@pytest.mark.parametrize("where", [KEY_S, KEY_DP, QUERY_S, QUERY_DP])
@pytest.mark.parametrize("d", [64, 128])
def test_sums_that_lack_the_last_step_are_not_stored(d, where):
    """Lists of two steps: the softmax is through both when the issuer gives up."""
    stall_and_recover(2, 250, d, where)


def stall_and_recover(H, N, d, where):
    n = W.cdiv(N, 64)
    mask = tsr.make_mask(tsr.UNIFORM, 1, H, N, d, bq=64, bk=64,
                         blocks=torch.ones((1, H, n, n), dtype=torch.uint8, device="cuda"))
    q, k, v = (t.cuda() for t in W.qkv(1, H, N, d, 3))
    do = W.qkv(1, H, N, d, 4)[0].cuda()
    out, lse = tsr.tsr_bsa_forward(q, k, v, tsr.tsr_plan(mask))
    plan = tsr.tsr_backward_plan(mask)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    want = tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan, workspace=ws)
    plan.device_status()
    plan.test_stall(where)
    got = [torch.full_like(q, float("nan")) for _ in range(3)]
    tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan, *got, workspace=ws)
    with pytest.raises(tsr.TsrError) as e:
        plan.device_status()
    assert e.value.status == 5
    plan.device_status()                                     # the error word was cleared
    # the other kind's items are whole; the stalled ones wrote nothing
    for g, w, bits in zip(got, want, (QUERY_S | QUERY_DP, KEY_S | KEY_DP, KEY_S | KEY_DP)):
        assert torch.all(torch.isnan(g)) if where & bits else torch.equal(g, w)
    plan.test_stall(0)
    again = tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan, workspace=ws)
    plan.device_status()
    assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_refusals():
    assert tsr.lib().tsr_backward_plan_test_stall(None, 1) == 1
    mask = tsr.make_mask(tsr.UNIFORM, 1, 1, 64, 64, bq=64, bk=64,
                         blocks=torch.ones((1, 1, 1, 1), dtype=torch.uint8, device="cuda"))
    plan = tsr.tsr_backward_plan(mask)
    for bad in (-1, 16):
        with pytest.raises(tsr.TsrError):
            plan.test_stall(bad)
