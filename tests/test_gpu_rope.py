"""Query / key norm with the position rotation, alone and with the append into a paged cache, against
the formulas in 64 bits.

Bar, per element: the kernel computes in fp32 (fewer than 64 roundings on the way from the inputs to a
pair's two products: sum of d squares, rsqrt, weight, rotation), so before its one rounding it is within
64 * 2^-24 = 2^-18 of (|a| + |b|), a and b the normed pair; the rounding adds eps/2 of the value, or half a
subnormal step (fp16: 2^-25).  Copies (V, untouched slots) are bit-exact.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sa():
    import quantized_attention_02_b200 as sa
    assert torch.cuda.is_available()
    return sa


def tables(rows, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * inv
    return a.cos().float().cuda(), a.sin().float().cuda()


def reference(x, w, cos, sin, eps, interleaved):
    """(value, size of what was added up for it) in 64 bits; cos, sin broadcast against x's leading dims."""
    y, rot = x.double(), 2 * cos.shape[-1]
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    c, s = cos.double(), sin.double()
    i = torch.arange(rot // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = y[..., ia], y[..., ib]
    out, size = y.clone(), y.abs()
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return out, size


def assert_close(got, ref, size):
    eps = torch.finfo(got.dtype).eps
    err = 2.0 ** -18 * size
    bound = err + eps / 2 * (ref.abs() + err) + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    d = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    assert (d <= bound).all(), float((d - bound).max())


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("B,N,Hq,Hk,d,rot,interleaved,norm", [
    (1, 1, 1, 1, 64, 64, False, True),
    (2, 7, 5, 3, 64, 16, True, True),
    (1, 33, 8, 2, 64, 32, False, False),
    (3, 130, 6, 1, 128, 128, True, False),
    (2, 257, 12, 4, 128, 128, False, True),
    (1, 19, 3, 0, 128, 48, False, True),   # queries alone, a rotation that is no power of two
    (2, 64, 48, 48, 64, 64, True, True),
    (1, 5, 2, 2, 128, 112, True, True),
    (1, 5, 2, 2, 128, 112, False, True),
])
def test_norm_rope(sa, dt, B, N, Hq, Hk, d, rot, interleaved, norm):
    g = torch.Generator().manual_seed(B * N + Hq + rot)
    qkv = (torch.randn(B, N, Hq + Hk, d, generator=g) * 3).to(DT[dt]).cuda()
    q = qkv[:, :, :Hq].transpose(1, 2)
    k = qkv[:, :, Hq:].transpose(1, 2) if Hk else None
    wq = wk = None
    if norm:
        wq, wk = (1 + 0.3 * torch.randn(2, d, generator=g)).to(DT[dt]).cuda()
    cos, sin = tables(500, rot)
    shared = N % 2 == 1
    pos = torch.randint(0, 500, (N,) if shared else (B, N), generator=g, dtype=torch.int32).cuda()
    before = qkv.clone()
    qo, ko = sa.qk_norm_rope(q, k, cos, sin, positions=pos, q_weight=wq, k_weight=wk, eps=1e-5, interleaved=interleaved)
    assert qo.is_contiguous() and torch.equal(qkv, before)
    at = pos.long().expand(B, N)
    c, s = cos[at][:, None], sin[at][:, None]
    assert_close(qo, *reference(q, wq, c, s, 1e-5, interleaved))
    if Hk:
        assert_close(ko, *reference(k, wk, c, s, 1e-5, interleaved))
    # positions left out: token n has position n
    qo, _ = sa.qk_norm_rope(q, k, cos, sin, q_weight=wq, k_weight=wk, eps=1e-5, interleaved=interleaved)
    assert_close(qo, *reference(q, wq, cos[:N], sin[:N], 1e-5, interleaved))


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_extremes(sa, interleaved):
    g = torch.Generator().manual_seed(5)
    q = torch.randn(1, 9, 4, 64, generator=g).half().cuda().transpose(1, 2)
    q[0, 0, 0] = 60000.0   # squares past fp16, not past fp32
    q[0, 1, 1] = 0.0       # a zero row stays zero (eps > 0)
    q[0, 2, 2] = 2.0 ** -24
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    cos, sin = tables(16, 64)
    want, size = reference(q, w, cos[:9], sin[:9], 1e-6, interleaved)
    sa.sage_qk_norm_rope(q, None, q, None, cos, sin, q_weight=w, interleaved=interleaved)
    assert_close(q, want, size)


def test_position_outside_the_table_gives_nan_rows_only(sa):
    q = torch.randn(1, 2, 4, 64, device="cuda").half()
    cos, sin = tables(8, 64)
    pos = torch.tensor([0, 8, -1, 7], dtype=torch.int32, device="cuda")
    o, _ = sa.qk_norm_rope(q, None, cos, sin, positions=pos)
    assert o[:, :, 1:3].isnan().all() and torch.isfinite(o[:, :, [0, 3]]).all()


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,d,rot,page,interleaved,norm", [
    (1, 4, 1, 64, 64, 16, False, True),
    (77, 14, 2, 64, 32, 16, True, True),
    (300, 8, 8, 128, 128, 32, False, True),
    (129, 6, 2, 128, 64, 256, False, False),
    (40, 32, 8, 128, 128, 128, False, True),
])
def test_append(sa, dt, heads_first, T, Hq, Hk, d, rot, page, interleaved, norm):
    g = torch.Generator().manual_seed(T + Hq)
    qkv = torch.randn(T, Hq + 2 * Hk, d, generator=g).to(DT[dt]).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    wq = wk = None
    if norm:
        wq, wk = (1 + 0.3 * torch.randn(2, d, generator=g)).to(DT[dt]).cuda()
    cos, sin = tables(1000, rot)
    pos = torch.randint(0, 1000, (T,), generator=g, dtype=torch.int32).cuda()
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:T].int()
    slots[T // 2::7] = -1
    slots[T // 3::11] = pages * page  # past the cache: not written either
    shape = (pages, Hk, page, d) if heads_first else (pages, page, Hk, d)
    kc = torch.randn(shape, generator=g).to(DT[dt]).cuda()
    vc = torch.randn(shape, generator=g).to(DT[dt]).cuda()
    kv, vv = (kc.transpose(1, 2), vc.transpose(1, 2)) if heads_first else (kc, vc)
    k0, v0 = kv.clone(), vv.clone()
    qo = sa.qk_norm_rope_append(q, k, v, cos, sin, pos, slots.cuda(), kv, vv, q_weight=wq, k_weight=wk,
                                interleaved=interleaved)
    c, s = cos[pos.long()][:, None], sin[pos.long()][:, None]
    assert_close(qo, *reference(q, wq, c, s, 1e-6, interleaved))
    kref, ksize = reference(k, wk, c, s, 1e-6, interleaved)
    kept = (slots >= 0) & (slots < pages * page)
    p, r = slots[kept].long() // page, slots[kept].long() % page
    assert_close(kv[p, r], kref[kept], ksize[kept])
    assert torch.equal(vv[p, r], v[kept])
    k0[p, r], v0[p, r] = kv[p, r], vv[p, r]
    assert torch.equal(kv, k0) and torch.equal(vv, v0)  # every other slot as it was


def test_no_tokens_and_refusals(sa):
    cos, sin = tables(8, 64)
    h = torch.float16
    e = torch.empty(1, 2, 0, 64, dtype=h, device="cuda")
    o, _ = sa.qk_norm_rope(e, None, cos, sin)
    assert o.shape == e.shape
    q = torch.randn(1, 2, 4, 64, device="cuda", dtype=h)
    with pytest.raises(ValueError):
        sa.qk_norm_rope(q.float(), None, cos, sin)
    with pytest.raises(ValueError):
        sa.qk_norm_rope(q, q.bfloat16(), cos, sin)
    with pytest.raises(ValueError):
        sa.qk_norm_rope(q, None, cos, sin[:4])
    with pytest.raises(ValueError):
        sa.qk_norm_rope(q, None, cos.half(), sin)
    with pytest.raises(ValueError):
        sa.qk_norm_rope(q, None, cos, sin, positions=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        sa.qk_norm_rope(q, None, cos, sin, q_weight=torch.ones(32, dtype=h, device="cuda"))
    with pytest.raises(ValueError):
        sa.qk_norm_rope(q.transpose(-1, -2), None, cos, sin)
    with pytest.raises(sa.SageError):  # a token stride that is no multiple of 8 elements
        sa.qk_norm_rope(torch.randn(4, 68, device="cuda", dtype=h)[:, :64][None, None], None, cos, sin)
    with pytest.raises(sa.SageError):  # more tokens than table rows, and no positions
        sa.qk_norm_rope(torch.randn(1, 1, 9, 64, device="cuda", dtype=h), None, cos, sin)
    cache = torch.zeros(2, 24, 1, 64, device="cuda", dtype=h)
    x = torch.randn(3, 1, 64, device="cuda", dtype=h)
    with pytest.raises(sa.SageError):  # page size
        sa.qk_norm_rope_append(x, x, x, cos, sin, None, torch.zeros(3, dtype=torch.int32, device="cuda"), cache, cache)


def test_side_stream_and_graph(sa):
    q = torch.randn(2, 4, 64, 128, device="cuda", dtype=torch.bfloat16)
    cos, sin = tables(64, 128)
    want, _ = sa.qk_norm_rope(q, None, cos, sin)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, _ = sa.qk_norm_rope(q, None, cos, sin, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.sage_qk_norm_rope(q, None, out, None, cos, sin)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_positions_that_are_no_tensor_are_refused(sa):
    cos, sin = tables(8, 64)
    q = torch.randn(1, 2, 4, 64, device="cuda", dtype=torch.float16)
    with pytest.raises(TypeError):
        sa.qk_norm_rope(q, None, cos, sin, positions=[0, 1, 2, 3])
    x = q[0].transpose(0, 1)
    cache = torch.zeros(2, 16, 2, 64, device="cuda", dtype=torch.float16)
    with pytest.raises(TypeError):
        sa.qk_norm_rope_append(x, x, x, cos, sin, [0, 1, 2, 3], torch.zeros(4, dtype=torch.int32, device="cuda"), cache, cache)
