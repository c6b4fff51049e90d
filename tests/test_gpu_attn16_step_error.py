"""The kernel for few query rows keeps twice the operand type's bits of each softmax weight.

It splits a weight into two 16-bit parts, so that its output is off by at most, to first order and in the names of
attn_reference (half = eps/2 of the type, A = sum_j p_j |v_j|, n keys):
  half |o|               its rounding to the output type
  half^2 A               what is left of a weight behind its two parts
  2 (ds + 2^-21) A       the weights themselves, in numerator and sum; 2^-21: twice the bound of ex2.approx, for the
                         rounding of a product with an fp32 factor as well (no polynomial here)
  (n + 32) 2^-24 A'      fp32 accumulation of n terms and the joining of parts, A' the largest |v|
  n 2^-31 A'             fp16 weights below the type's normal range
A weight rounded once would be off by half A, and the sums below are made to show it."""
import pytest
import torch

from attn_reference import attend

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sa():
    import quantized_attention_02_b200 as sa
    assert torch.cuda.is_available()
    yield sa
    assert sa.sage_last_device_error() == 0


def bar(dt, q, k, v, ref, A, sm_scale):
    half, n = torch.finfo(dt).eps / 2, k.shape[1]
    ds = 2.0 ** -16 * sm_scale * (q.double().abs() @ k.double().abs().transpose(-1, -2)).amax(-1, keepdim=True)
    most = v.double().abs().amax(1, keepdim=True)
    out = half * ref.abs() + (half ** 2 + 2 * (ds + 2.0 ** -21)) * A + ((n + 32) * 2.0 ** -24 + n * 2.0 ** -31) * most
    return 1.02 * out + (2.0 ** -24 if dt == torch.float16 else 0.0)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hk,tokens,n", [(1, 1, 1, 1, 2), (1, 4, 1, 1, 130), (2, 8, 2, 4, 400), (1, 16, 1, 1, 1000),
                                              (40, 4, 2, 2, 700), (300, 4, 4, 1, 300)])
def test_opposite_values_with_weights_that_round_alike(sa, dt, d, B, Hq, Hk, tokens, n):
    # Half of the keys have weight 1 and value 1, the others weight p a little below 1 and value -1.  p = 1 - 0.45 half
    # is nearest to 1 in the operand type, so that weights rounded once cancel to 0, where o = (1 - p) / (1 + p).
    half = torch.finfo(DT[dt]).eps / 2
    q = torch.zeros(B, Hq, tokens, d, dtype=DT[dt], device="cuda")
    q[..., 0] = 1.0
    k = torch.zeros(B, Hk, n, d, dtype=DT[dt], device="cuda")
    k[:, :, 1::2, 0] = -0.45 * half
    v = torch.ones(B, Hk, n, d, dtype=DT[dt], device="cuda")
    v[:, :, 1::2] = -1.0
    o = sa.sageattn_cross(q, k, v, sm_scale=1.0)
    kk, vv = (x[0].repeat_interleave(Hq // Hk, 0) for x in (k, v))
    ref, _, A = attend(q[0], kk, vv, torch.ones(tokens, n, dtype=torch.bool, device="cuda"), 1.0)
    limit = bar(DT[dt], q[0], kk, vv, ref, A, 1.0)
    if n % 2 == 0:  # the bar tells the two apart
        assert (limit < ref.abs() / 1.5).all()
    assert ((o.double() - ref).abs() <= limit).all(), ((o.double() - ref).abs() / limit).max().item()


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hk,tokens,lengths", [(32, 8, 1, [1, 17, 128, 129, 500, 3000]), (6, 2, 5, [700, 5000]),
                                                  (16, 1, 1, [9000]), (3, 3, 16, [40, 1000])])
def test_random_weights(sa, dt, d, Hq, Hk, tokens, lengths):
    g = torch.Generator(device="cuda").manual_seed(sum(lengths))
    B, Nk = len(lengths), max(lengths)
    q = (torch.randn(B, Hq, tokens, d, generator=g, device="cuda") * 1.5).to(DT[dt])
    k, v = torch.randn(2, B, Hk, Nk, d, generator=g, device="cuda").to(DT[dt])
    o = sa.sageattn_cross(q, k, v, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    for b, n in enumerate(lengths):
        kk, vv = (x[b, :, :n].repeat_interleave(Hq // Hk, 0) for x in (k, v))
        ref, _, A = attend(q[b], kk, vv, torch.ones(tokens, n, dtype=torch.bool, device="cuda"), d ** -0.5)
        err = (o[b].double() - ref).abs() / bar(DT[dt], q[b], kk, vv, ref, A, d ** -0.5)
        assert err.max().item() <= 1, (b, err.max().item())
