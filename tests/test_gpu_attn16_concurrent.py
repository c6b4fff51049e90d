"""Calls of the paged and the cross attention at the same time: host threads, captured graphs on streams of their own, a
process whose first call is under capture."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from test_gpu_paged_attn import problem, run

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NEW = [1, 20, 200]  # tokens: the kernel for few rows, for one tile, for pairs of tiles; all join parts


@pytest.fixture(scope="module")
def sa():
    import quantized_attention_02_b200 as sa
    assert torch.cuda.is_available()
    yield sa
    assert sa.sage_last_device_error() == 0


def problems(sa):
    ps = [problem([(n, 6000), (1, 3000)], 8, 2, 128, 64, torch.bfloat16, seed=n)[0] for n in NEW]
    want = [run(sa, p, True, 0.09) for p in ps]
    torch.cuda.synchronize()
    return ps, want


def test_host_threads(sa):
    ps, want = problems(sa)
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for n in range(30):
                j = (i + n) % len(ps)
                got = run(sa, ps[j], True, 0.09)
                stream.synchronize()
                if not torch.equal(got, want[j]):
                    wrong.append((i, n))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_graphs_replayed_at_the_same_time(sa):
    ps, want = problems(sa)
    graphs, outs = [], []
    for p in ps * 2:
        o = torch.full_like(p["q"], 99.0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sa.sage_paged_attn(p["q"], p["k_cache"], p["v_cache"], o, p["page_table"], p["cu_q"], p["kv_len"], True, 0.09)
        graphs.append(graph)
        outs.append(o)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for o in outs:
            o.fill_(99.0)
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want * 2))


def test_stream_handles(sa):
    (p, *_), (want, *_) = problems(sa)
    args = (p["q"], p["k_cache"], p["v_cache"], p["page_table"], p["cu_q"], p["kv_len"])
    stream = torch.cuda.Stream()
    for handle in (stream, stream.cuda_stream, 0):
        o = sa.sageattn_paged(*args, sm_scale=0.09, stream=handle)
        torch.cuda.synchronize()
        rows = int(p["cu_q"][-1])
        assert torch.equal(o[:rows], want[:rows])


FIRST_CALL = """
import sys, torch
sys.path.insert(0, {root!r})
import quantized_attention_02_b200 as sa
g = torch.Generator().manual_seed(1)
q = torch.randn(2, 8, {nq}, 64, generator=g).half().cuda()
k, v = torch.randn(2, 2, 2, 3000, 64, generator=g).half().cuda()
cos = torch.ones(300, 32, device="cuda")
sin = torch.zeros(300, 32, device="cuda")
o, r = torch.zeros_like(q), torch.zeros_like(q)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    sa.sage_qk_norm_rope(q, None, r, None, cos, sin)
    sa.sage_cross_attn(r, k, v, o, None, 0.125)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(r, q)
assert torch.equal(o, sa.sageattn_cross(q, k, v)), "differs"
assert sa.sage_last_device_error() == 0
print("same")
"""


@pytest.mark.parametrize("nq", [1, 30, 200])
def test_the_first_call_of_a_process_under_capture(nq):
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=ROOT, nq=nq)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
