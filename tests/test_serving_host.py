"""Refusals of the serving operators, ahead of any CUDA call (no GPU needed): the C ABI's statuses for
bad sizes, types, strides, pages and pointers, and the binding's errors for tensors off the GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def sa():
    from quantized_attention_02_b200 import build
    build.build()
    import quantized_attention_02_b200 as sa
    return sa


FAKE, ODD = 0x1000, 0x1008  # never dereferenced: the calls below fail validation first


def strides(sa, b=8192, h=1024, n=128):
    return sa.SageStrides(b, h, n)


def rope(sa, **kw):
    st = strides(sa)
    a = dict(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, qs=st, ks=st, qos=st, kos=st, wq=None, wk=None, cos=FAKE, sin=FAKE,
             pos=None, per_batch=0, B=1, Hq=4, Hk=2, N=8, d=128, rot=128, rows=64, il=0, eps=1e-6, dtype=sa.SAGE_BF16,
             stream=None)
    a.update(kw)
    return sa.get_lib().sage_qk_norm_rope(*a.values())


def append(sa, **kw):
    st = strides(sa)
    a = dict(q=FAKE, k=FAKE, v=FAKE, qo=FAKE, kc=FAKE, vc=FAKE, qs=st, ks=st, vs=st, qos=st, kcs=st, vcs=st, wq=None,
             wk=None, cos=FAKE, sin=FAKE, pos=None, slots=FAKE, T=8, Hq=4, Hk=2, d=128, rot=128, rows=64, pages=4,
             page=16, il=0, eps=1e-6, dtype=sa.SAGE_BF16, stream=None)
    a.update(kw)
    return sa.get_lib().sage_qk_norm_rope_append(*a.values())


INVALID, UNSUPPORTED = -1, -2

ROPE_REFUSED = [
    (dict(q=None), INVALID), (dict(q=ODD), INVALID), (dict(qo=None), INVALID), (dict(cos=None), INVALID),
    (dict(sin=ODD), INVALID), (dict(wq=ODD), INVALID), (dict(k=None), INVALID), (dict(qs=None), INVALID),
    (dict(B=-1), INVALID), (dict(N=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hk=-1), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(rot=0), INVALID), (dict(rot=24), INVALID), (dict(rot=144), INVALID),
    (dict(rows=0), INVALID), (dict(rows=7), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(dtype=2), INVALID), (dict(B=1 << 20, N=1 << 12, rows=1 << 12), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", ROPE_REFUSED, ids=lambda v: str(v))
def test_norm_rope_refuses(sa, kw, status):
    assert rope(sa, **kw) == status


@pytest.mark.parametrize("field,value", [("b", 12), ("h", 4), ("n", 0), ("n", -128)])
def test_norm_rope_refuses_strides(sa, field, value):
    st = strides(sa)
    setattr(st, field, value)
    for name in ("qs", "ks", "qos", "kos"):
        assert rope(sa, B=2, **{name: st}) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(slots=None), INVALID), (dict(v=None), INVALID), (dict(kc=ODD), INVALID), (dict(Hk=0), INVALID),
    (dict(T=-1), INVALID), (dict(page=0), INVALID), (dict(pages=0), INVALID), (dict(page=8), UNSUPPORTED),
    (dict(page=48), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(pages=1 << 27, page=16), UNSUPPORTED),
    (dict(T=1 << 29), INVALID), (dict(T=1 << 29, pos=FAKE), UNSUPPORTED), (dict(d=32), UNSUPPORTED),
], ids=lambda v: str(v))
def test_append_refuses(sa, kw, status):
    assert append(sa, **kw) == status


def test_no_tokens_is_no_work(sa):
    assert rope(sa, N=0, q=None, qo=None, k=None, ko=None) == 0
    assert rope(sa, B=0) == 0
    assert append(sa, T=0, q=None, slots=None) == 0


def test_binding_refuses_host_tensors(sa):
    x = torch.zeros(1, 2, 3, 64, dtype=torch.float16)
    t = torch.zeros(8, 32)
    with pytest.raises(ValueError):
        sa.qk_norm_rope(x, None, t, t)
    with pytest.raises(ValueError):
        sa.qk_norm_rope_append(x[0], x[0], x[0], t, t, None, torch.zeros(2, dtype=torch.int32), x, x)
    with pytest.raises(TypeError):
        sa.qk_norm_rope(None, None, t, t)


def test_strides_struct_matches_the_header(sa):
    assert ctypes.sizeof(sa.SageStrides) == 24
    assert [n for n, _ in sa.SageStrides._fields_] == ["b", "h", "n"]


def paged(sa, **kw):
    st = strides(sa)
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, o=FAKE, qs=st, kcs=st, vcs=st, os=st, table=FAKE, cu=FAKE, len=FAKE, B=2, T=8,
             Hq=4, Hk=2, d=128, pages=4, page=16, width=2, causal=1, scale=0.1, dtype=sa.SAGE_F16, stream=None)
    a.update(kw)
    return sa.get_lib().sage_paged_attn(*a.values())


def cross(sa, **kw):
    st = strides(sa)
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, qs=st, ks=st, vs=st, os=st, len=None, B=2, Hq=4, Hk=2, Nq=8, Nk=9, d=128,
             scale=0.1, dtype=sa.SAGE_F16, stream=None)
    a.update(kw)
    return sa.get_lib().sage_cross_attn(*a.values())


ATTN_REFUSED = [
    (dict(q=None), INVALID), (dict(q=ODD), INVALID), (dict(o=None), INVALID), (dict(o=ODD), INVALID),
    (dict(B=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID), (dict(Hk=3), INVALID),
    (dict(Hq=130, Hk=1), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(dtype=2), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
]


@pytest.mark.parametrize("kw,status", ATTN_REFUSED + [
    (dict(kc=None), INVALID), (dict(vc=ODD), INVALID), (dict(table=None), INVALID), (dict(cu=None), INVALID),
    (dict(len=None), INVALID), (dict(T=-1), INVALID), (dict(pages=0), INVALID), (dict(width=-1), INVALID),
    (dict(page=8), UNSUPPORTED), (dict(page=100), UNSUPPORTED), (dict(page=512), UNSUPPORTED),
    (dict(width=(1 << 20) + 1), UNSUPPORTED), (dict(B=(1 << 24) + 1), UNSUPPORTED), (dict(T=1 << 29), UNSUPPORTED),
], ids=lambda v: str(v))
def test_paged_attn_refuses(sa, kw, status):
    assert paged(sa, **kw) == status


@pytest.mark.parametrize("kw,status", ATTN_REFUSED + [
    (dict(k=None), INVALID), (dict(v=ODD), INVALID), (dict(Nq=-1), INVALID), (dict(Nk=-1), INVALID),
    (dict(Nq=1 << 29), UNSUPPORTED), (dict(Nk=(1 << 24) + 1), UNSUPPORTED),
], ids=lambda v: str(v))
def test_cross_attn_refuses(sa, kw, status):
    assert cross(sa, **kw) == status


@pytest.mark.parametrize("field,value,status", [("b", 12, INVALID), ("h", 4, INVALID), ("n", 0, INVALID),
                                                ("n", -128, INVALID), ("b", 1 << 40, UNSUPPORTED)])
def test_attention_refuses_strides(sa, field, value, status):
    st = strides(sa)
    setattr(st, field, value)
    for name in ("qs", "ks", "vs"):
        assert cross(sa, **{name: st}) == status
    for name in ("kcs", "vcs"):
        assert paged(sa, **{name: st}) == status


def test_attention_without_tokens_is_no_work(sa):
    assert paged(sa, T=0, q=None, o=None) == 0 and paged(sa, B=0, table=None, cu=None, len=None) == 0
    assert cross(sa, Nq=0, q=None, o=None) == 0 and cross(sa, B=0) == 0


def test_paged_attn_refuses_more_sequences_than_its_waits_allow(sa):
    assert paged(sa, B=(1 << 20) + 1) == UNSUPPORTED


def test_the_unsupported_status_names_the_page_sizes(sa):
    assert append(sa, page=48) == UNSUPPORTED and "page" in sa.sage_status_string(UNSUPPORTED)
