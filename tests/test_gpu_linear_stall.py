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


@pytest.mark.parametrize("T,K,M", [(2, 256, 512), (5, 1160, 264), (72, 1352, 3560), (700, 264, 1544), (1038, 1776, 8),
                                   (2593, 1176, 1712), (200, 4096, 264), (20011, 64, 64)])
def test_a_stalled_product_stores_nothing(T, K, M):
    """What a product that gave up has not computed is not stored either: its outputs stay as
    they were, whole tiles, tiles cut along k and clusters' tiles alike."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    x, w, r, dout = rand(T, K), rand(M, K), rand(T, M), rand(T, M)
    want = tsr.tsr_linear(x, w, activation="silu", residual=r, pre=True)
    grads = tsr.tsr_linear_backward(dout, x, w, activation="silu", pre=want[1])
    kept = lambda *like: [torch.full_like(t, 7.0) for t in like]
    out, pre = kept(*want)
    dx, dw, db = kept(*grads)
    tsr.tsr_linear_device_status()
    stall(1)
    try:
        tsr.tsr_linear(x, w, activation="silu", residual=r, out=out, pre=pre)
        tsr.tsr_linear_backward(dout, x, w, activation="silu", pre=want[1], dx=dx, dweight=dw, dbias=db)
        with pytest.raises(tsr.TsrError) as e:
            tsr.tsr_linear_device_status()
        assert e.value.status == 5
    finally:
        stall(0)
    assert all((t == 7.0).all() for t in (out, pre, dx, dw))
    assert torch.equal(db, grads[2])                           # summed before the products
    again = [*tsr.tsr_linear(x, w, activation="silu", residual=r, out=out, pre=pre),
             *tsr.tsr_linear_backward(dout, x, w, activation="silu", pre=want[1], dx=dx, dweight=dw, dbias=db)]
    assert all(torch.equal(a, b) for a, b in zip(again, (*want, *grads)))
    tsr.tsr_linear_device_status()
