"""Random problems for the paged and the cross attention against the formula in 64 bits: groups of 1 to 128 heads, empty
and ragged lengths, every page size, unused rows full of NaN."""
import random

import pytest
import torch

import test_gpu_cross_attn as cross
import test_gpu_paged_attn as paged

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def sa():
    import quantized_attention_02_b200 as sa
    assert torch.cuda.is_available()
    yield sa
    assert sa.sage_last_device_error() == 0


def heads(rng):
    group, Hk = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 8, 12, 16, 17, 24, 48, 64, 65, 128]), rng.choice([1, 2, 3, 8])
    return group, 1 if group * Hk > 256 else Hk


@pytest.mark.parametrize("seed", range(12))
def test_paged(sa, seed):
    rng = random.Random(seed)
    done = 0
    while done < 8:
        group, Hk = heads(rng)
        d, dt, page, causal = rng.choice([64, 128]), rng.choice(TYPES), rng.choice([16, 32, 64, 128, 256]), rng.random() < .7
        B, new, keys = rng.choice([1, 2, 3, 5, 9, 20, 60, 200]), rng.choice([1, 1, 2, 4, 17, 40, 130, 400]), rng.choice([1, 16, 130, 700, 3001, 9000])
        seqs = [(rng.choice([0, 1, 1, new, rng.randint(0, new)]), rng.choice([0, 1, keys, rng.randint(0, keys)])) for _ in range(B)]
        if B * keys * new * group * Hk > 3e8 or B * keys * Hk * d > 1e8 or not any(n for n, _ in seqs):
            continue
        p, k, v, cu = paged.problem(seqs, group * Hk, Hk, d, page, dt, seed=100 * seed + done, heads_first=rng.random() < .5)
        o = paged.run(sa, p, causal, 0.1)
        paged.check(o, p, seqs, k, v, cu, causal, 0.1)
        assert (o[cu[-1]:] == 99).all()
        done += 1


@pytest.mark.parametrize("seed", range(12))
def test_cross(sa, seed):
    rng = random.Random(1000 + seed)
    done = 0
    while done < 8:
        group, Hk = heads(rng)
        d, dt = rng.choice([64, 128]), rng.choice(TYPES)
        B, Nq = rng.choice([1, 2, 3, 10, 40]), rng.choice([1, 2, 5, 16, 17, 33, 64, 127, 128, 129, 200, 500, 1000])
        Nk = rng.choice([1, 2, 15, 64, 127, 128, 129, 226, 257, 640, 1500, 5000])
        if B * Nq * Nk * group * Hk > 3e8 or B * Nk * Hk * d > 1e8:
            continue
        lengths = None if rng.random() < .4 else [rng.choice([0, 1, Nk, rng.randint(0, Nk)]) for _ in range(B)]
        g = torch.Generator(device="cuda").manual_seed(100 * seed + done)
        q = (torch.randn(B, Nq, group * Hk, d, generator=g, device="cuda") * 2).to(dt).transpose(1, 2)
        kv = torch.randn(B, Nk, 2, Hk, d, generator=g, device="cuda").to(dt)
        for b, n in enumerate(lengths or []):
            kv[b, n:] = float("nan")
        k, v = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
        o = sa.sageattn_cross(q, k, v, None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"), 0.1)
        cross.check(o, q, k, v, lengths, 0.1)
        done += 1
