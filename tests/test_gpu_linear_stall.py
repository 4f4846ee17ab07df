"""The bounded waits of a linear layer's products: a product whose issuer stops gives up and
says so, the context stays usable, and the next product is whole.  Each kind of tile and
kernel (pairs of CTAs, cut along k or not; clusters for few tokens)."""
import pytest
import torch

import block_sparse_attention_tsr_gb300 as tsr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tsr.build()
    tsr.lib()


def stall(on):
    assert tsr.lib().tsr_linear_test_stall(on) == 0


@pytest.mark.parametrize("T,K,M", [(2, 256, 512), (5, 1160, 264), (72, 1352, 3560), (700, 264, 1544), (1038, 1776, 8),
                                   (2593, 1176, 1712)])
def test_a_stalled_product_gives_up(T, K, M):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    want = tsr.tsr_linear(x, w)
    tsr.tsr_linear_device_status()
    stall(1)
    try:
        tsr.tsr_linear(x, w)
        with pytest.raises(tsr.TsrError) as e:
            tsr.tsr_linear_device_status()
        assert e.value.status == 5
        tsr.tsr_linear_backward(want, x, w)
        with pytest.raises(tsr.TsrError) as e:
            tsr.tsr_linear_device_status()
        assert e.value.status == 5
    finally:
        stall(0)
    assert torch.equal(tsr.tsr_linear(x, w), want)
    tsr.tsr_linear_device_status()


def test_refusal():
    assert tsr.lib().tsr_linear_test_stall(2) == 1
