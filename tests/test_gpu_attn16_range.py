"""Values at the end of fp16's range: an output is a mean of values and stays among them, whichever kernel ran."""
import pytest
import torch

from attn_reference import assert_attention, attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    import quantized_attention_02_b200 as sa
    assert torch.cuda.is_available()
    yield sa
    assert sa.sage_last_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens,batch,n", [(1, 2, 400), (40, 2, 400), (300, 2, 400), (300, 160, 400),  # as one part
                                            (1, 2, 5000), (40, 2, 5000), (300, 2, 5000)])  # joined from parts
def test_a_mean_of_the_largest_values_stays_finite(sa, tokens, batch, n, d):
    # One key of a later tile has most of the weight, 2^0.7 to 2^7.2 times that of the first tile's largest: a weight
    # whose 16-bit rounding is off by up to 2^-11, and with it the mean.
    g = torch.Generator(device="cuda").manual_seed(tokens + n)
    q = torch.zeros(batch, 4, tokens, d, dtype=torch.float16, device="cuda")
    q[..., 0] = (0.1 + 0.9 * torch.rand(batch, 4, tokens, generator=g, device="cuda")).half()
    k = torch.zeros(batch, 2, n, d, dtype=torch.float16, device="cuda")
    k[..., 0] = -60.0
    k[:, :, 0, 0], k[:, :, 300, 0] = 0.0, 5.0
    sign = 1 - 2 * (torch.arange(d, device="cuda") % 2)
    v = (65504.0 * sign).half().expand(batch, 2, n, d).contiguous()
    o = sa.sageattn_cross(q, k, v, sm_scale=1.0)
    assert o.isfinite().all()
    seen = torch.ones(tokens, n, dtype=torch.bool, device="cuda")
    for h in range(4):
        assert_attention(o[0, h][None], *attend(q[0, h][None], k[0, h // 2][None], v[0, h // 2][None], seen, 1.0))


@pytest.mark.parametrize("tokens,batch,n", [(1, 2, 400), (40, 2, 400), (300, 2, 400), (300, 160, 400), (40, 2, 5000), (300, 2, 5000)])
def test_infinite_values_stay_infinite(sa, tokens, batch, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    q = torch.randn(batch, 4, tokens, 64, generator=g, device="cuda").half()
    k, v = torch.randn(2, batch, 2, n, 64, generator=g, device="cuda").half()
    v[0, 0, 17, 5], v[0, 1, 300, 9] = float("inf"), float("-inf")
    o = sa.sageattn_cross(q, k, v, sm_scale=0.1)
    assert (o[0, :2, :, 5] == float("inf")).all() and (o[0, 2:, :, 9] == float("-inf")).all()
    rest = o.clone()
    rest[0, :2, :, 5] = rest[0, 2:, :, 9] = 0
    assert rest.isfinite().all()
