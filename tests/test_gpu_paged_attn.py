"""Attention over a paged cache against the formula in 64 bits (bar: attn_reference)."""
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


def problem(seqs, Hq, Hk, d, page, dt, seed=0, heads_first=False, spare=3, tail=5):
    """seqs: (new tokens, keys) of each sequence.  Unused pages, rows past a sequence's end and table
    entries past its pages hold NaN or nonsense; `tail` tokens stand behind the last sequence."""
    g = torch.Generator().manual_seed(seed)
    count = [-(-kv // page) for _, kv in seqs]
    total = sum(count) + spare
    perm = torch.randperm(total, generator=g)
    width = max(count + [1]) + 1
    table = torch.full((len(seqs), width), 2 ** 31 - 1, dtype=torch.int32)
    shape = (total, Hk, page, d) if heads_first else (total, page, Hk, d)
    kc, vc = torch.full(shape, float("nan")), torch.full(shape, float("nan"))
    kc, vc = (x.transpose(1, 2) if heads_first else x for x in (kc, vc))
    keys, values, at = [], [], 0
    for b, (_, kv) in enumerate(seqs):
        pages = perm[at:at + count[b]]
        at += count[b]
        table[b, :count[b]] = pages.int()
        k, v = torch.randn(2, kv, Hk, d, generator=g)
        j = torch.arange(kv)
        kc[pages[j // page], j % page], vc[pages[j // page], j % page] = k, v
        keys.append(k.to(dt).cuda())
        values.append(v.to(dt).cuda())
    cu = [0]
    for nq, _ in seqs:
        cu.append(cu[-1] + nq)
    q = (torch.randn(cu[-1] + tail, Hq, d, generator=g) * 1.5).to(dt).cuda()
    def cache(x):
        x = x.to(dt)
        return (x.transpose(1, 2).contiguous().cuda().transpose(1, 2)) if heads_first else x.cuda()
    return dict(q=q, k_cache=cache(kc), v_cache=cache(vc), page_table=table.cuda(),
                cu_q=torch.tensor(cu, dtype=torch.int32).cuda(),
                kv_len=torch.tensor([kv for _, kv in seqs], dtype=torch.int32).cuda()), keys, values, cu


def check(o, p, seqs, keys, values, cu, causal, sm_scale):
    group = p["q"].shape[1] // p["k_cache"].shape[2]
    for b, (nq, kv) in enumerate(seqs):
        if nq == 0:
            continue
        got = o[cu[b]:cu[b + 1]].transpose(0, 1)
        if kv == 0:
            assert (got == 0).all()
            continue
        i, j = torch.arange(nq, device="cuda")[:, None], torch.arange(kv, device="cuda")[None]
        seen = (j <= kv - nq + i) if causal else torch.ones(nq, kv, dtype=torch.bool, device="cuda")
        k, v = (x[b].transpose(0, 1).repeat_interleave(group, 0) for x in (keys, values))
        assert_attention(got, *attend(p["q"][cu[b]:cu[b + 1]].transpose(0, 1), k, v, seen, sm_scale))


def run(sa, p, causal, sm_scale):
    """Into an output whose every row is marked: (o, mark)."""
    o = torch.full_like(p["q"], 99.0)
    sa.sage_paged_attn(p["q"], p["k_cache"], p["v_cache"], o, p["page_table"], p["cu_q"], p["kv_len"], causal, sm_scale)
    return o


SEQS = {
    "one_key": [(1, 1)],
    "steps": [(1, 1), (1, 16), (1, 17), (1, 127), (1, 128), (1, 129), (1, 500), (1, 0)],
    "long_step": [(1, 6000)],
    "two_long_steps": [(1, 9000), (1, 300)],
    "chunk": [(100, 100)],
    "chunks": [(64, 200), (1, 77), (0, 50), (200, 200), (129, 1000), (3, 3)],
    "chunk_far": [(70, 5000)],
    "more_new_than_keys": [(40, 10), (300, 150), (5, 0)],
    "many_long_steps": [(1, 6000 - 100 * i) for i in range(40)] * 2,
    "long_chunks": [(200, 3000), (150, 5000), (1, 4000)] * 6,
    "long_speculative": [(30, 3000)] * 20 + [(1, 2000)] * 5,
    "two_or_three": [(2, 900), (3, 1500), (0, 10), (1, 3), (2, 1)] * 3,
    "one_chunk_among_none": [(0, 100)] * 30 + [(29, 800)] + [(0, 5)] * 10,
    "idle": [(0, 100), (0, 0)],
    "many_steps": [(1, 1 + 53 * i % 900) for i in range(700)],
    "many_chunks": [(64 - i % 5, 64 + 13 * i % 300) for i in range(300)],
    "many": [(1 + i % 3, 1 + 37 * i % 400) for i in range(500)],
}


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", list(SEQS))
@pytest.mark.parametrize("Hq,Hk,d,page,heads_first", [(8, 2, 128, 64, False), (7, 1, 64, 16, True)])
def test_paged(sa, dt, causal, name, Hq, Hk, d, page, heads_first):
    seqs = SEQS[name]
    p, keys, values, cu = problem(seqs, Hq, Hk, d, page, DT[dt], seed=len(name), heads_first=heads_first)
    o = run(sa, p, causal, d ** -0.5)
    check(o, p, seqs, keys, values, cu, causal, d ** -0.5)
    assert (o[cu[-1]:] == 99).all()  # rows behind the last sequence


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("Hq,Hk,d", [(1, 1, 64), (4, 4, 128), (12, 4, 64), (40, 8, 128), (128, 1, 64)])
def test_pages_and_groups(sa, page, Hq, Hk, d):
    seqs = [(1, 700), (150, 390), (17, 256), (2, 1300)]
    p, keys, values, cu = problem(seqs, Hq, Hk, d, page, torch.bfloat16, seed=page + Hq, heads_first=Hq % 8 == 0)
    check(run(sa, p, True, 0.09), p, seqs, keys, values, cu, True, 0.09)


def test_wide_table_splits_by_the_real_length(sa):
    # a table for 65536 keys, a sequence of 130: the parts of the key axis follow the length on the device
    seqs = [(1, 130), (1, 64)]
    p, keys, values, cu = problem(seqs, 8, 2, 128, 64, torch.float16)
    wide = torch.full((2, 1024), -1, dtype=torch.int32, device="cuda")
    wide[:, :p["page_table"].shape[1]] = p["page_table"]
    p["page_table"] = wide
    check(run(sa, p, True, 0.09), p, seqs, keys, values, cu, True, 0.09)


def test_bad_pages_read_as_zeros_and_lengths_are_clamped(sa):
    seqs = [(1, 64), (1, 64)]
    p, keys, values, cu = problem(seqs, 2, 1, 64, 16, torch.float16)
    p["page_table"][0, 1] = -5
    p["page_table"][1, 2] = 10 ** 6
    p["kv_len"][1] = 10 ** 6  # more than its 5 table entries hold: 80 keys, the last page bad as well
    keys[0][16:32] = values[0][16:32] = 0
    keys[1][32:48] = values[1][32:48] = 0
    zero = torch.zeros(16, 1, 64, dtype=torch.float16, device="cuda")
    keys[1], values[1] = torch.cat((keys[1], zero)), torch.cat((values[1], zero))
    check(run(sa, p, True, 0.125), p, [(1, 64), (1, 80)], keys, values, cu, True, 0.125)
    p["kv_len"][:] = -3
    assert (run(sa, p, True, 0.125)[:2] == 0).all()


@pytest.mark.parametrize("cu", [[0, 300, 100, 400], [400, 0, 0, 50], [-7, 90, 10 ** 6, 3]])
@pytest.mark.parametrize("Hq,Hk", [(4, 4), (8, 2), (64, 1)])
def test_cu_q_that_is_not_ascending_stays_inside(sa, cu, Hq, Hk):
    p, *_ = problem([(100, 100), (200, 200), (100, 300)], Hq, Hk, 64, 32, torch.float16, tail=0)
    p["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    buf = torch.full((600, Hq, 64), 3.0, dtype=torch.float16, device="cuda")
    o = buf[100:500]
    sa.sage_paged_attn(p["q"], p["k_cache"], p["v_cache"], o, p["page_table"], p["cu_q"], p["kv_len"], True, 0.125)
    torch.cuda.synchronize()
    assert (buf[:100] == 3).all() and (buf[500:] == 3).all()


def test_no_pages_at_all(sa):
    p, *_ = problem([(1, 64), (3, 64)], 2, 1, 64, 16, torch.float16)
    p["page_table"] = p["page_table"][:, :0].contiguous()
    o = run(sa, p, True, 0.125)
    assert (o[:4] == 0).all() and (o[4:] == 99).all()


def test_strided_queries_and_output(sa):
    seqs = [(30, 200), (1, 90)]
    p, keys, values, cu = problem(seqs, 6, 2, 64, 32, torch.bfloat16)
    fused = torch.randn(p["q"].shape[0], 10, 64, device="cuda").bfloat16()
    fused[:, 2:8] = p["q"]
    p["q"] = fused[:, 2:8]
    buf = torch.full((p["q"].shape[0], 8, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    o = buf[:, 1:7]
    sa.sage_paged_attn(p["q"], p["k_cache"], p["v_cache"], o, p["page_table"], p["cu_q"], p["kv_len"], True, 0.125)
    check(o, p, seqs, keys, values, cu, True, 0.125)
    assert (buf[:, 0] == 5).all() and (buf[:, 7] == 5).all()


@pytest.mark.parametrize("new", [1, 20, 200])  # the kernel for few rows, for one tile, for pairs of tiles
def test_same_bits_again_and_under_capture(sa, new):
    seqs = [(new, 7000), (1, 3000), (4, 500)]
    p, keys, values, cu = problem(seqs, 8, 2, 128, 64, torch.bfloat16)
    want = run(sa, p, True, 0.09)
    o = torch.zeros_like(want)
    args = (p["q"], p["k_cache"], p["v_cache"], o, p["page_table"], p["cu_q"], p["kv_len"], True, 0.09)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sa.sage_paged_attn(*args)
        graphs.append(graph)
    for graph in graphs * 2:
        o.fill_(99.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [sa.sageattn_paged(*args[:3], *args[4:], stream=s) for s in streams for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(x[:cu[-1]], want[:cu[-1]]) for x in got)
    # lengths that changed between replays are seen
    p["kv_len"][0] = 1000
    keys[0], values[0] = keys[0][:1000], values[0][:1000]
    graphs[0].replay()
    check(o, p, [(new, 1000), (1, 3000), (4, 500)], keys, values, cu, True, 0.09)


def test_offsets_past_32_bits(sa):
    # a cache of more than 2^32 bytes and more than 2^31 elements: the last pages
    page, Hk, d = 256, 8, 128
    pages = (1 << 31) // (page * Hk * d) + 40
    cache = torch.zeros(2, pages, page, Hk, d, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(4)
    kv = 1000
    ids = [pages - 1, 2, pages - 3, pages - 2]
    k, v = torch.randn(2, kv, Hk, d, generator=g).bfloat16().cuda()
    j = torch.arange(kv, device="cuda")
    at = torch.tensor(ids, device="cuda")[j // page]
    cache[0][at, j % page], cache[1][at, j % page] = k, v
    q = torch.randn(1, Hk, d, generator=g).bfloat16().cuda()
    o = sa.sageattn_paged(q, cache[0], cache[1], torch.tensor([ids], dtype=torch.int32, device="cuda"),
                          torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                          torch.tensor([kv], dtype=torch.int32, device="cuda"))
    seen = torch.ones(1, kv, dtype=torch.bool, device="cuda")
    assert_attention(o.transpose(0, 1), *attend(q.transpose(0, 1), k.transpose(0, 1), v.transpose(0, 1), seen, d ** -0.5))


def test_no_tokens_and_refusals(sa):
    p, *_ = problem([(1, 64)], 2, 1, 64, 16, torch.float16)
    e = sa.sageattn_paged(p["q"][:0], p["k_cache"], p["v_cache"], p["page_table"], p["cu_q"], p["kv_len"])
    assert e.shape[0] == 0
    args = (p["k_cache"], p["v_cache"], p["page_table"], p["cu_q"], p["kv_len"])
    with pytest.raises(ValueError):
        sa.sageattn_paged(p["q"].bfloat16(), *args)
    with pytest.raises(ValueError):
        sa.sageattn_paged(p["q"], p["k_cache"], p["v_cache"][1:], *args[2:])
    with pytest.raises(ValueError):
        sa.sageattn_paged(p["q"], *args[:2], p["page_table"].long(), *args[3:])
    with pytest.raises(ValueError):
        sa.sageattn_paged(p["q"], *args[:3], p["cu_q"][:1], p["kv_len"])
    with pytest.raises(sa.SageError):
        sa.sageattn_paged(p["q"], p["k_cache"][:, :8], p["v_cache"][:, :8], *args[2:])


# ------------------------------------------------------------------ the operators together
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_prompt_in_chunks_then_single_tokens(sa, dt):
    """A prompt enters the cache in chunks and is followed by single tokens; every step's attention equals
    that of the whole sequence at once, computed in 64 bits from the cached keys and values."""
    T, Hq, Hk, d, page = 300, 8, 2, 64, 32
    g = torch.Generator().manual_seed(11)
    qkv = torch.randn(T, Hq + 2 * Hk, d, generator=g).to(DT[dt]).cuda()
    w = (1 + 0.2 * torch.randn(2, d, generator=g)).to(DT[dt]).cuda()
    inv = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    a = torch.arange(512, dtype=torch.float64)[:, None] * inv
    cos, sin = a.cos().float().cuda(), a.sin().float().cuda()
    pages = -(-T // page)
    order = torch.randperm(pages + 4, generator=g)[:pages].int()
    table = order[None].cuda()
    kc, vc = (torch.full((pages + 4, page, Hk, d), float("nan"), dtype=DT[dt], device="cuda") for _ in range(2))
    q_all, o_all, at = [], [], 0
    for n in (128, 100, 7, *[1] * (T - 235)):
        pos = torch.arange(at, at + n, dtype=torch.int32)
        slots = (order[(pos // page).long()] * page + pos % page).int().cuda()
        new = qkv[at:at + n]
        q = sa.qk_norm_rope_append(new[:, :Hq], new[:, Hq:Hq + Hk], new[:, Hq + Hk:], cos, sin, pos.cuda(), slots, kc, vc,
                                   q_weight=w[0], k_weight=w[1])
        at += n
        o_all.append(sa.sageattn_paged(q, kc, vc, table, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                                       torch.tensor([at], dtype=torch.int32, device="cuda")))
        q_all.append(q)
    j = torch.arange(T)
    k, v = (c[order[j // page].long(), j % page] for c in (kc, vc))
    assert torch.equal(v, qkv[:, Hq + Hk:])
    whole_q, whole_k = sa.qk_norm_rope(qkv[None, :, :Hq].transpose(1, 2), qkv[None, :, Hq:Hq + Hk].transpose(1, 2), cos,
                                       sin, q_weight=w[0], k_weight=w[1])
    assert torch.equal(whole_k[0].transpose(0, 1), k) and torch.equal(whole_q[0].transpose(0, 1), torch.cat(q_all))
    seen = torch.ones(T, T, dtype=torch.bool, device="cuda").tril()
    k, v = (x.transpose(0, 1).repeat_interleave(Hq // Hk, 0) for x in (k, v))
    assert_attention(torch.cat(o_all).transpose(0, 1), *attend(whole_q[0], k, v, seen, d ** -0.5))


def test_video_block(sa):
    """Norm and rotation, the framework's self attention, then cross attention to padded text states."""
    g = torch.Generator().manual_seed(12)
    B, N, H, d, Nk = 2, 500, 4, 64, 77
    qkv = torch.randn(B, N, 3 * H, d, generator=g).half().cuda()
    inv = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    a = torch.arange(N, dtype=torch.float64)[:, None] * inv
    w = torch.ones(d, dtype=torch.float16, device="cuda")
    q, k = sa.qk_norm_rope(qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:2 * H].transpose(1, 2), a.cos().float().cuda(),
                           a.sin().float().cuda(), q_weight=w, k_weight=w, interleaved=True)
    v = qkv[:, :, 2 * H:].transpose(1, 2).contiguous()
    x = sa.sageattn(q, k, v)
    full = torch.ones(N, N, dtype=torch.bool, device="cuda")
    for b in range(B):
        want, _, _ = attend(q[b], k[b], v[b], full, d ** -0.5)
        assert torch.nn.functional.cosine_similarity(x[b].double().flatten(), want.flatten(), 0) > 0.999
    text = torch.randn(2, B, H, Nk, d, generator=g).half().cuda()
    lengths = torch.tensor([77, 30], dtype=torch.int32, device="cuda")
    o = sa.sageattn_cross(x, text[0], text[1], key_len=lengths)
    for b, n in enumerate((77, 30)):
        seen = torch.ones(N, n, dtype=torch.bool, device="cuda")
        assert_attention(o[b], *attend(x[b], text[0][b, :, :n], text[1][b, :, :n], seen, d ** -0.5))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seqs", [
    [(150, 1000)] + [(150, 0)] * 20 + [(150, 2000)],
    [(700, 300)] * 5 + [(400, 1)] * 40 + [(30, 1000)],  # causal: most tokens see no key
    [(260, 0)] * 300 + [(260, 500)] + [(260, 0)] * 100 + [(1, 77)],
], ids=["empty_between", "more_new_than_keys", "many_empty"])
def test_long_runs_of_items_without_keys(sa, seqs, d, causal):
    p, keys, values, cu = problem(seqs, 4, 2, d, 64, torch.bfloat16)
    o = run(sa, p, causal, 0.1)
    assert sa.sage_last_device_error() == 0
    check(o, p, seqs, keys, values, cu, causal, 0.1)
    assert (o[cu[-1]:] == 99.0).all()


# ------------------------------------------------------------------ many sequences, nearly all of them empty
@pytest.mark.parametrize("B", [31, 32, 33, 64, 65, 1024, 1025, 1056, 1057, 7000])
@pytest.mark.parametrize("rows", ["tile", "pair"])
def test_few_among_many_sequences(sa, B, rows):
    # the place of a slot's sequence is looked up among B: first, last and some in between have tokens
    G, d = 8, 64
    # the average rows of a sequence choose the kernel: 17 to 128 of them, or more
    total = -(-B * (40 if rows == "tile" else 140) // G)
    at = sorted({0, B // 3, B // 2, B // 2 + 1, B - 1})
    seqs = [(0, 10)] * B
    for n, b in enumerate(at):
        seqs[b] = (total // len(at) + (total % len(at) if n == 0 else 0), 65 + 100 * n)
    p, keys, values, cu = problem(seqs, G, 1, d, 64, torch.float16, seed=B)
    o = run(sa, p, False, 0.1)
    check(o, p, seqs, keys, values, cu, False, 0.1)
    assert (o[cu[-1]:] == 99).all()


def test_a_walk_past_many_empty_sequences_is_short(sa):
    # 20000 sequences of which the first has all tokens; a walk that looks at all sequences for each slot takes 30 ms
    B, T = 20000, 322500
    q = torch.zeros(T, 8, 64, dtype=torch.float16, device="cuda")
    cache = torch.ones(2, 64, 1, 64, dtype=torch.float16, device="cuda")
    cu = torch.full((B + 1,), T, dtype=torch.int32, device="cuda")
    cu[0] = 0
    kv = torch.full((B,), 100, dtype=torch.int32, device="cuda")
    table = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
    times = []
    for _ in range(4):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        o = sa.sageattn_paged(q, cache, cache, table, cu, kv, False)
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end))
    assert (o == 1).all()
    assert min(times) < 10


@pytest.mark.parametrize("new", [1, 20, 100])
def test_heads_first_cache_with_head_strides_past_32_bits(sa, new):
    # [Hk][pages][page][d] in memory: 2^31 elements and more from one head to the next
    page, Hk, Hq, d, kv = 256, 2, 8, 64, 500
    pages = (1 << 31) // (page * d) + 2
    caches = [torch.empty(Hk, pages, page, d, dtype=torch.float16, device="cuda").permute(1, 2, 0, 3) for _ in range(2)]
    assert caches[0].stride(2) >= 1 << 31
    ids = torch.tensor([pages - 1, pages - 2], device="cuda")
    k, v = torch.randn(2, kv, Hk, d, generator=torch.Generator().manual_seed(new)).half().cuda()
    j = torch.arange(kv, device="cuda")
    for cache, x in zip(caches, (k, v)):
        cache[ids[j // page], j % page] = x
    q = torch.randn(new, Hq, d, generator=torch.Generator().manual_seed(new)).half().cuda()
    o = sa.sageattn_paged(q, *caches, ids.int()[None], torch.tensor([0, new], dtype=torch.int32, device="cuda"),
                          torch.tensor([kv], dtype=torch.int32, device="cuda"))
    seen = j[None] <= kv - new + torch.arange(new, device="cuda")[:, None]
    k, v = (x.transpose(0, 1).repeat_interleave(Hq // Hk, 0) for x in (k, v))
    assert_attention(o.transpose(0, 1), *attend(q.transpose(0, 1), k, v, seen, d ** -0.5))


# ------------------------------------------------------------------ a cu_q that is not ascending, on every path
PATHS = {  # sequences as in problem(), Hq, Hk: rows of an average sequence (tokens x group) choose the kernel
    "step": ([(16, 300), (16, 1000), (16, 100)], 4, 4),             # 16
    "step_groups": ([(4, 300), (4, 700), (4, 100)], 16, 4),         # 16 in groups of four
    "step_many": ([(n % 5, 40 + n) for n in range(300)], 4, 2),     # 4 on average, more than one scan of the sequences
    "tile": ([(30, 300), (30, 200), (40, 400)], 4, 2),              # 67, the key axis in one part
    "tile_split": ([(30, 1500), (30, 1000), (40, 2000)], 4, 2),     # 67, in parts that are joined
    "tile_many": ([(20 + n % 9, 50 + n) for n in range(60)], 4, 2),  # 48
    "pair_cut": ([(100, 100), (200, 200), (100, 300)], 4, 2),       # 267, few items
    "pair_whole": ([(100, 100), (200, 200), (100, 300)], 384, 6),   # 8533, 618 items: dealt out whole
    "pair_many": ([(80 + n % 9, 50 + n) for n in range(60)], 16, 8),  # 168, more items than four per SM
}


@pytest.mark.parametrize("order", ["falling", "outside", "mixed"])
@pytest.mark.parametrize("path", list(PATHS))
def test_any_cu_q_stays_inside(sa, path, order):
    seqs, Hq, Hk = PATHS[path]
    p, keys, values, cu = problem(seqs, Hq, Hk, 64, 32, torch.float16, tail=0)
    T, B = cu[-1], len(seqs)
    good = run(sa, p, True, 0.125)
    r = torch.Generator().manual_seed(B)
    p["cu_q"] = {
        "falling": torch.linspace(T, 0, B + 1).int(),
        "outside": torch.tensor([-2 ** 31, 2 ** 31 - 1, -7, T + 3], dtype=torch.int32).repeat(B)[:B + 1],
        "mixed": torch.randint(-T // 4, T + T // 4, (B + 1,), generator=r, dtype=torch.int32),
    }[order].cuda()
    buf = torch.full((T + 200, Hq, 64), 3.0, dtype=torch.float16, device="cuda")
    for causal in (True, False):
        sa.sage_paged_attn(p["q"], p["k_cache"], p["v_cache"], buf[100:T + 100], p["page_table"], p["cu_q"], p["kv_len"],
                           causal, 0.125)
    torch.cuda.synchronize()
    assert (buf[:100] == 3).all() and (buf[T + 100:] == 3).all()
    assert sa.sage_last_device_error() == 0
    p["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    assert torch.equal(run(sa, p, True, 0.125), good)
