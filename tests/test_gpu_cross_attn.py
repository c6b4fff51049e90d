"""Cross attention against the formula in 64 bits (bar: attn_reference)."""
import pytest
import torch

from attn_reference import assert_attention, attend

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sa():
    import quantized_attention_02_b200 as sa
    assert torch.cuda.is_available()
    yield sa
    assert sa.sage_last_device_error() == 0


def check(o, q, k, v, lengths, sm_scale):
    group = q.shape[1] // k.shape[1]
    for b in range(q.shape[0]):
        n = k.shape[2] if lengths is None else lengths[b]
        kb, vb = (x[b, :, :n].repeat_interleave(group, 0) for x in (k, v))
        if n == 0:
            assert (o[b] == 0).all()
            continue
        assert_attention(o[b], *attend(q[b], kb, vb, torch.ones(q.shape[2], n, dtype=torch.bool, device="cuda"), sm_scale))


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("B,Hq,Hk,Nq,Nk,d,lengths", [
    (1, 1, 1, 1, 1, 64, None),
    (2, 4, 4, 130, 100, 64, [100, 1]),
    (2, 4, 2, 300, 129, 128, [129, 128]),
    (3, 6, 2, 77, 257, 128, [0, 257, 130]),      # one entry without keys; groups of three
    (1, 2, 1, 1000, 640, 64, None),
    (2, 7, 1, 33, 1000, 64, [999, 5]),           # seven heads share a key head, odd query count
    (4, 8, 8, 1, 1500, 64, [1500, 700, 64, 1]),  # single tokens
    (1, 32, 8, 1, 5000, 128, None),              # single token, key axis split
    (1, 2, 2, 257, 9000, 128, None),             # few tiles, long states: split with pairs of tiles
    (20, 32, 8, 1, 2500, 128, None),             # more CTAs than SMs, no split: long walks through the rings
    (40, 16, 8, 1, 5001, 64, None),
    (20, 16, 8, 40, 2500, 128, None),            # one query tile per sequence: 80 rows
    (25, 12, 6, 33, 3001, 64, None),
    (3, 5, 1, 3, 1000, 128, [1000, 0, 17]),      # fifteen rows of five heads
    (300, 2, 1, 2, 70, 64, None),                # many short sequences
    (2, 32, 16, 700, 4100, 128, None),
    (4, 40, 40, 1000, 226, 64, [226, 64, 128, 1]),  # more items than four per SM: dealt out whole
    (4, 80, 40, 500, 333, 128, [333, 0, 77, 129]),
    (2, 128, 1, 3, 300, 64, [300, 17]),          # the widest group: one token per tile
    (1, 96, 1, 5, 700, 128, None),
])
def test_cross(sa, dt, B, Hq, Hk, Nq, Nk, d, lengths):
    g = torch.Generator().manual_seed(B + Hq + Nq + Nk)
    q = (torch.randn(B, Hq, Nq, d, generator=g) * 2).to(DT[dt]).cuda()
    kv = torch.randn(B, Nk, 2, Hk, d, generator=g).to(DT[dt]).cuda()
    k, v = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)  # strided views of one projection
    key_len = None
    if lengths is not None:
        key_len = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lengths):  # padding may hold anything
            kv[b, n:, 0] = float("nan")
            kv[b, n:, 1] = float("inf")
    o = sa.sageattn_cross(q, k, v, key_len=key_len)
    check(o, q, k, v, lengths, d ** -0.5)


@pytest.mark.parametrize("Nq,Nk", [(1, 0), (200, 0)])
def test_no_keys_at_all(sa, Nq, Nk):
    q = torch.randn(2, 4, Nq, 64, device="cuda").half()
    k = torch.empty(2, 2, Nk, 64, device="cuda", dtype=torch.float16)
    assert (sa.sageattn_cross(q, k, k) == 0).all()


@pytest.mark.parametrize("std", [0.0, 1e-3, 12.0])
def test_flat_and_peaked_scores(sa, std):
    # from equal weights to rows dominated by one key (offsets that move, weights that underflow)
    g = torch.Generator().manual_seed(3)
    q = (torch.randn(1, 2, 300, 128, generator=g) * std).half().cuda()
    k = (torch.randn(1, 2, 1111, 128, generator=g) * max(std, 1)).half().cuda()
    v = (torch.randn(1, 2, 1111, 128, generator=g) + 3).half().cuda()
    check(sa.sageattn_cross(q, k, v, sm_scale=0.3), q, k, v, None, 0.3)


def test_ascending_scores_move_the_offset(sa):
    # scores grow along the keys, so every tile raises the maximum: the accumulator is rescaled each time
    k = torch.zeros(1, 1, 1500, 64)
    k[..., 0] = torch.linspace(-300, 300, 1500)
    q = torch.zeros(1, 1, 200, 64)
    q[..., 0] = torch.linspace(-2, 2, 200)[None, None]
    v = torch.randn(1, 1, 1500, 64, generator=torch.Generator().manual_seed(1))
    for dt in DT.values():
        a, b, c = (x.to(dt).cuda() for x in (q, k, v))
        check(sa.sageattn_cross(a, b, c, sm_scale=0.5), a, b, c, None, 0.5)


def test_output_view_and_rows_around_it(sa):
    g = torch.Generator().manual_seed(9)
    q = torch.randn(2, 4, 150, 64, generator=g).bfloat16().cuda()
    k, v = torch.randn(2, 2, 4, 333, 64, generator=g).bfloat16().cuda()
    buf = torch.full((2, 152, 6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    o = buf[:, 1:151, 1:5].transpose(1, 2)
    sa.sage_cross_attn(q, k, v, o, None, 0.125)
    check(o, q, k, v, None, 0.125)
    assert (buf[:, 0] == 7).all() and (buf[:, 151] == 7).all() and (buf[:, :, 0] == 7).all() and (buf[:, :, 5] == 7).all()


@pytest.mark.parametrize("Nq", [1, 40, 300])  # the kernel for few rows, for one tile, for pairs of tiles
def test_streams_and_graph(sa, Nq):
    g = torch.Generator().manual_seed(2)
    q = torch.randn(1, 8, Nq, 128, generator=g).half().cuda()
    k, v = torch.randn(2, 1, 8, 4000, 128, generator=g).half().cuda()
    want = sa.sageattn_cross(q, k, v)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [sa.sageattn_cross(q, k, v, stream=s) for s in (s1, s2) * 10]  # overlapping calls, own workspaces
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    o = torch.zeros_like(q)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sa.sage_cross_attn(q, k, v, o, None, 128 ** -0.5)
        graphs.append(graph)
    for graph in graphs:
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)


def test_binding_refuses(sa):
    q = torch.randn(1, 4, 8, 64, device="cuda").half()
    k = torch.randn(1, 2, 9, 64, device="cuda").half()
    with pytest.raises(ValueError):
        sa.sageattn_cross(q, k.bfloat16(), k)
    with pytest.raises(ValueError):
        sa.sageattn_cross(q, k, k[:, :, :8])
    with pytest.raises(ValueError):
        sa.sageattn_cross(q, k, k, key_len=torch.tensor([9], device="cuda"))
    with pytest.raises(ValueError):
        sa.sageattn_cross(q, k.transpose(-1, -2), k.transpose(-1, -2))
    with pytest.raises(sa.SageError):
        sa.sageattn_cross(q[:, :3], k, k)
    with pytest.raises(sa.SageError):
        sa.sageattn_cross(q, k[:, :1].expand(1, 2, 9, 64), k)  # heads that share memory: stride 0
    with pytest.raises(sa.SageError):
        sa.sageattn_cross(q, k, k, sm_scale=0.0)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("B,Hq,Hk,Nq,Nk,d,lengths", [
    (3, 128, 8, 128, 5000, 64, [977, 0, 5000]),   # 64 pairs of query tiles without a key between others, cut axis
    (3, 128, 8, 128, 5000, 128, [977, 0, 5000]),
    (9, 32, 16, 500, 700, 128, [0, 0, 700, 0, 0, 0, 0, 0, 1]),
    (40, 40, 40, 300, 200, 64, [200 if b in (0, 17, 38) else 0 for b in range(40)]),  # dealt out whole
    (40, 40, 40, 300, 200, 128, [200 if b in (0, 17, 38) else 0 for b in range(40)]),
])
def test_long_runs_of_items_without_keys(sa, dt, B, Hq, Hk, Nq, Nk, d, lengths):
    g = torch.Generator().manual_seed(7)
    q = torch.randn(B, Nq, Hq, d, generator=g).to(DT[dt]).cuda().transpose(1, 2)
    k, v = torch.randn(2, B, Hk, Nk, d, generator=g).to(DT[dt]).cuda()
    o = sa.sageattn_cross(q, k, v, torch.tensor(lengths, dtype=torch.int32, device="cuda"), 0.2)
    assert sa.sage_last_device_error() == 0
    check(o, q, k, v, lengths, 0.2)
