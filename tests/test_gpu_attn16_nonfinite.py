"""Scores that are not finite among the keys a token sees, in each of the three 16-bit attention kernels.

By the formula a score of NaN or +inf makes the token's whole row NaN, and a score of -inf has no weight, at
whatever place of a key tile it stands; where every score is -inf the row is 0, as without a key."""
import math

import pytest
import torch

from attn_reference import assert_attention, attend

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
# tokens of a sequence -> kernel, with two heads per key head: few rows, one tile, pairs of tiles (cut, dealt out whole)
KERNELS = {"step": (1, 2), "tile": (40, 2), "pair": (300, 2), "pair_whole": (300, 160)}


@pytest.fixture(scope="module")
def sa():
    import quantized_attention_02_b200 as sa
    assert torch.cuda.is_available()
    yield sa
    assert sa.sage_last_device_error() == 0


def problem(kernel, dt, d, n, seed):
    """One batch entry per case: q [B, Hq, N, d], k, v [B, Hk, n, d] (Hk = Hq / 2)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    tokens, batch = KERNELS[kernel]
    q = torch.randn(batch, 4, tokens, d, generator=g, device="cuda").to(DT[dt])
    k, v = torch.randn(2, batch, 2, n, d, generator=g, device="cuda").to(DT[dt])
    return q, k, v


def same_as_without(o, q, k, v, left_out):
    """Rows of one batch entry and query head against the formula without the keys of `left_out` ([n] bool)."""
    seen = (~left_out)[None].expand(q.shape[0], -1)
    k = torch.where(left_out[:, None], torch.zeros_like(k), k)
    assert_attention(o[None], *attend(q[None], k[None], v[None], seen, 0.1))


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), math.inf])
def test_one_key_at_every_place_of_a_tile(sa, value, dt, d, kernel):
    n = 900
    q, k, v = problem(kernel, dt, d, n, 1)
    q[..., 0] = q[..., 0].abs() + 0.5  # the infinite channel gives +inf
    clean = sa.sageattn_cross(q, k, v, sm_scale=0.1)
    for place in [0, 5, 127, *range(384, 400), *range(468, 484), *range(576, 592), 895, 899]:
        bad = k.clone()
        bad[0, 0, place, 0] = value
        o = sa.sageattn_cross(q, bad, v, sm_scale=0.1)
        assert o[0, :2].isnan().all(), place  # both heads of the key head
        assert torch.equal(o[0, 2:], clean[0, 2:]) and torch.equal(o[1:], clean[1:]), place


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_scores_of_minus_infinity_have_no_weight(sa, dt, d, kernel):
    n = 900
    q, k, v = problem(kernel, dt, d, n, 2)
    q[..., 0] = q[..., 0].abs() + 0.5
    gone = torch.zeros(2, n, dtype=torch.bool, device="cuda")
    gone[0, 0:300] = True  # the row's first tiles as a whole, and a part of one
    gone[1, 5::16] = gone[1, 14::16] = gone[1, 15::16] = True
    k[0, 0, gone[0], 0] = k[0, 1, gone[1], 0] = -math.inf
    o = sa.sageattn_cross(q, k, v, sm_scale=0.1)
    for h in range(4):
        same_as_without(o[0, h], q[0, h], k[0, h // 2], v[0, h // 2], gone[h // 2])


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_every_score_minus_infinity(sa, dt, d, kernel):
    q, k, v = problem(kernel, dt, d, 900, 3)
    q[..., 0] = q[..., 0].abs() + 0.5
    clean = sa.sageattn_cross(q, k, v, sm_scale=0.1)
    k[0, 0, :, 0] = -math.inf
    o = sa.sageattn_cross(q, k, v, sm_scale=0.1)
    assert (o[0, :2] == 0).all()
    assert torch.equal(o[0, 2:], clean[0, 2:]) and torch.equal(o[1:], clean[1:])
    for place in (3, 398, 527, 899):  # and one of them NaN
        bad = k.clone()
        bad[0, 0, place, 0] = math.nan
        assert sa.sageattn_cross(q, bad, v, sm_scale=0.1)[0, :2].isnan().all(), place


@pytest.mark.parametrize("group,tokens", [(3, 30), (7, 100), (5, 300)])  # tiles with rows past the last token's head
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_groups_that_do_not_fill_a_tile(sa, dt, group, tokens):
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(2, 2 * group, tokens, 64, generator=g, device="cuda").to(DT[dt])
    k, v = torch.randn(2, 2, 2, 700, 64, generator=g, device="cuda").to(DT[dt])
    clean = sa.sageattn_cross(q, k, v, sm_scale=0.1)
    k[1, 1, 398, 3] = math.nan
    o = sa.sageattn_cross(q, k, v, sm_scale=0.1)
    assert o[1, group:].isnan().all()
    assert torch.equal(o[0], clean[0]) and torch.equal(o[1, :group], clean[1, :group])
