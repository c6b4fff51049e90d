"""Cases of the serving operators around the attention forward pass: per-head query / key norm with the position
rotation (alone, or with the append into a paged cache), attention of a chunk of new tokens over a paged cache, and
cross attention to an encoder's states.

``run`` computes them from elementary torch operations in 32 bits, or with this repository's operators where ``own``
is true; ``exact`` gives the same results from the operators' definitions in 64 bits.
"""
import math
import random

import torch

own = False

_DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
_EPS = 1e-6


def listed():
    return [
        # one decoding step of eight requests: the latency of a single small pass
        {"name": "rope_append_step", "op": "rope_append", "dtype": "bf16", "T": 8, "Hq": 32, "Hk": 8, "d": 128,
         "rot": 128, "interleaved": False, "norm": True, "page": 64, "table": 8192},
        # a prompt of 8192 tokens entering the cache
        {"name": "rope_append_prompt", "op": "rope_append", "dtype": "bf16", "T": 8192, "Hq": 32, "Hk": 8, "d": 128,
         "rot": 128, "interleaved": False, "norm": True, "page": 64, "table": 32768},
        # video transformer block, projection layout in, the attention's [B, H, N, d] layout out
        {"name": "rope_heads_video", "op": "rope_heads", "dtype": "fp16", "B": 2, "N": 16384, "Hq": 48, "Hk": 48,
         "d": 64, "rot": 64, "interleaved": True, "norm": True},
        # partial rotation, no norm, odd token count
        {"name": "rope_heads_partial", "op": "rope_heads", "dtype": "bf16", "B": 3, "N": 1237, "Hq": 24, "Hk": 6,
         "d": 64, "rot": 32, "interleaved": False, "norm": False},
        # single tokens of a few short requests with an odd group of heads: latency
        {"name": "paged_step_short", "op": "paged", "dtype": "fp16", "B": 4, "nq": 1, "kv": 700, "ragged": True,
         "Hq": 14, "Hk": 2, "d": 64, "page": 16},
        # single tokens of a batch of requests of mixed lengths
        {"name": "paged_step_batch", "op": "paged", "dtype": "bf16", "B": 48, "nq": 1, "kv": 8192, "ragged": True,
         "Hq": 32, "Hk": 8, "d": 128, "page": 64},
        # one request far into a long context
        {"name": "paged_step_long", "op": "paged", "dtype": "bf16", "B": 1, "nq": 1, "kv": 131072, "ragged": False,
         "Hq": 32, "Hk": 8, "d": 128, "page": 128},
        # a mixed step: prompts' chunks and single tokens together, lengths that end inside pages and tiles
        {"name": "paged_mixed", "op": "paged", "dtype": "bf16", "B": 16, "nq": 333, "kv": 4099, "ragged": True,
         "Hq": 32, "Hk": 4, "d": 128, "page": 16},
        # a chunk of a long prompt
        {"name": "paged_chunk", "op": "paged", "dtype": "bf16", "B": 1, "nq": 2048, "kv": 16384, "ragged": False,
         "Hq": 32, "Hk": 8, "d": 128, "page": 64},
        # a decoder's single tokens against the encoder's states
        {"name": "cross_step", "op": "cross", "dtype": "fp16", "B": 16, "Nq": 1, "Nk": 1500, "ragged": True,
         "Hq": 16, "Hk": 16, "d": 64},
        # video tokens against padded text states
        {"name": "cross_video", "op": "cross", "dtype": "fp16", "B": 2, "Nq": 16384, "Nk": 226, "ragged": True,
         "Hq": 48, "Hk": 48, "d": 64},
        # long queries against long states, shared heads
        {"name": "cross_long", "op": "cross", "dtype": "bf16", "B": 2, "Nq": 4096, "Nk": 6001, "ragged": False,
         "Hq": 32, "Hk": 8, "d": 128},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_append", "rope_heads", "paged", "paged", "cross", "cross"])
    d = rng.choice([64, 128])
    hk = rng.choice([1, 2, 4, 6, 8])
    case = {"op": op, "dtype": rng.choice(["fp16", "bf16"]), "Hk": hk, "d": d}
    if op == "rope_append":
        case.update(T=_log(rng, 1, 8192), Hq=hk * rng.choice([1, 3, 4, 8]), rot=rng.choice([32, 64, d]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.6, page=rng.choice([16, 32, 64, 128, 256]),
                    table=rng.choice([8192, 32768]))
    elif op == "rope_heads":
        case.update(B=rng.choice([1, 2]), N=_log(rng, 1, 16384), Hq=hk * rng.choice([1, 3, 4, 8]),
                    rot=rng.choice([32, 64, d]), interleaved=rng.random() < 0.5, norm=rng.random() < 0.6)
        if case["Hq"] + hk > 48:
            case["Hq"] = hk * 3
    elif op == "paged":
        chunk = rng.random() < 0.5
        b = _log(rng, 1, 12 if chunk else 64)
        case.update(B=b, nq=_log(rng, 2, 700) if chunk else 1, kv=_log(rng, 16, 32768 // b if chunk else 262144 // b),
                    ragged=rng.random() < 0.7, Hq=hk * rng.choice([1, 3, 4, 7, 8]), page=rng.choice([16, 32, 64, 128, 256]))
        case["nq"] = max(1, min(case["nq"], case["kv"]))
    else:
        b = _log(rng, 1, 16)
        case.update(B=b, Nq=_log(rng, 1, 8192 // b), Nk=_log(rng, 1, 6001), ragged=rng.random() < 0.5,
                    Hq=hk * rng.choice([1, 3, 4]))
    return case


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """Chunk lengths and cache lengths of a paged case: a function of the case alone."""
    r = random.Random("%(B)d %(nq)d %(kv)d %(Hq)d %(Hk)d %(d)d %(page)d" % case)
    kv = [r.randint(max(1, case["kv"] // 4), case["kv"]) if case["ragged"] else case["kv"] for _ in range(case["B"])]
    kv[0] = case["kv"]
    nq = [r.randint(1, case["nq"]) if case["ragged"] else case["nq"] for _ in kv]
    nq[0] = case["nq"]
    return [min(a, b) for a, b in zip(nq, kv)], kv


def _key_lengths(case):
    r = random.Random("%(B)d %(Nq)d %(Nk)d %(Hq)d %(Hk)d %(d)d" % case)
    n = [r.randint(max(1, case["Nk"] // 4), case["Nk"]) for _ in range(case["B"])]
    n[0] = case["Nk"]
    return n


def _angles(rows, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * inv
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, d, hq, hk = _DTYPES[case["dtype"]], case["d"], case["Hq"], case["Hk"]

    def randn(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    s = {"op": case["op"], "case": case}
    if case["op"] in ("rope_append", "rope_heads"):
        s["eps"] = _EPS
        s["interleaved"] = case["interleaved"]
        s["wq"] = s["wk"] = None
        if case["norm"]:
            s["wq"], s["wk"] = 1 + 0.2 * randn(d), 1 + 0.2 * randn(d)
    if case["op"] == "rope_append":
        t, page = case["T"], case["page"]
        qkv = randn(t, hq + 2 * hk, d)  # one projection's output, used in place
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["cos"], s["sin"] = _angles(case["table"], case["rot"])
        s["positions"] = torch.randint(0, case["table"], (t,), generator=g, device="cuda", dtype=torch.int32)
        pages = -(-t // page) + 8
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:t].to(torch.int32)
        slots[torch.rand(t, generator=g, device="cuda") < 1 / 64] = -1  # padded tokens
        s["slots"] = slots
        s["k_cache"], s["v_cache"] = randn(pages, page, hk, d), randn(pages, page, hk, d)
    elif case["op"] == "rope_heads":
        b, n = case["B"], case["N"]
        qkv = randn(b, n, hq + 2 * hk, d)
        s["q"], s["k"] = qkv[:, :, :hq].transpose(1, 2), qkv[:, :, hq:hq + hk].transpose(1, 2)
        s["cos"], s["sin"] = _angles(n, case["rot"])
    elif case["op"] == "paged":
        nq, kv = _lengths(case)
        page = case["page"]
        count = [-(-n // page) for n in kv]
        width = max(count)
        total = sum(count) + 3
        perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        used = torch.arange(width, device="cuda")[None, :] < torch.tensor(count, device="cuda")[:, None]
        table = torch.full((len(kv), width), -1, dtype=torch.int32, device="cuda")
        table[used] = perm[:sum(count)]
        s["page_table"], s["kv_len"] = table, ints(kv)
        s["cu_q"] = ints([sum(nq[:i]) for i in range(len(nq) + 1)])
        s["q"] = randn(sum(nq), hq, d, std=1.5)
        s["k_cache"], s["v_cache"] = randn(total, page, hk, d), randn(total, page, hk, d)
    else:
        b = case["B"]
        s["q"] = randn(b, hq, case["Nq"], d, std=1.5)
        kv = randn(b, case["Nk"], 2, hk, d)  # one projection of the encoder's states
        s["k"], s["v"] = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
        s["key_len"] = ints(_key_lengths(case)) if case["ragged"] else None
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        import quantized_attention_02_b200 as sa
        if s["op"] == "rope_append":
            q = sa.qk_norm_rope_append(s["q"], s["k"], s["v"], s["cos"], s["sin"], s["positions"], s["slots"],
                                       s["k_cache"], s["v_cache"], q_weight=s["wq"], k_weight=s["wk"], eps=s["eps"],
                                       interleaved=s["interleaved"])
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if s["op"] == "rope_heads":
            q, k = sa.qk_norm_rope(s["q"], s["k"], s["cos"], s["sin"], q_weight=s["wq"], k_weight=s["wk"],
                                   eps=s["eps"], interleaved=s["interleaved"])
            return {"q": q, "k": k}
        if s["op"] == "paged":
            return sa.sageattn_paged(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["cu_q"], s["kv_len"],
                                     causal=True)
        return sa.sageattn_cross(s["q"], s["k"], s["v"], key_len=s["key_len"])
    if s["op"] == "rope_append":
        cos, sin = s["cos"][s["positions"]][:, None], s["sin"][s["positions"]][:, None]  # [T, 1, rot/2]
        q = _norm_rope(s["q"], s["wq"], cos, sin, s["eps"], s["interleaved"])
        k = _norm_rope(s["k"], s["wk"], cos, sin, s["eps"], s["interleaved"])
        kept = s["slots"] >= 0
        page = s["k_cache"].shape[1]
        p, o = s["slots"][kept].long() // page, s["slots"][kept].long() % page
        s["k_cache"][p, o] = k[kept]
        s["v_cache"][p, o] = s["v"][kept]
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "rope_heads":
        cos, sin = s["cos"], s["sin"]  # [N, rot/2]
        return {"q": _norm_rope(s["q"], s["wq"], cos, sin, s["eps"], s["interleaved"]).contiguous(),
                "k": _norm_rope(s["k"], s["wk"], cos, sin, s["eps"], s["interleaved"]).contiguous()}
    if s["op"] == "paged":
        q, cu, kv = s["q"], s["cu_q"].long(), s["kv_len"].long()
        b, (t, hq, d) = kv.numel(), q.shape
        nq = cu[1:] - cu[:-1]
        most = min(t, s["case"]["nq"])
        i = torch.arange(most, device=q.device)
        rows = (cu[:-1, None] + i).clamp(max=t - 1)  # [B, most]
        k = s["k_cache"][s["page_table"].clamp(min=0).long()].flatten(1, 2)  # [B, L, Hk, d]
        v = s["v_cache"][s["page_table"].clamp(min=0).long()].flatten(1, 2)
        j = torch.arange(k.shape[1], device=q.device)
        seen = (j < kv[:, None])[:, None] & (j <= (kv - nq)[:, None, None] + i[:, None])  # [B, most, L]
        o = _attention(q[rows].transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), seen)  # [B, Hq, most, d]
        out = torch.empty_like(q)
        there = i < nq[:, None]
        out[rows[there]] = o.transpose(1, 2)[there]
        return out
    k, v = s["k"], s["v"]
    j = torch.arange(k.shape[2], device=k.device)
    length = torch.full((k.shape[0],), k.shape[2], device=k.device) if s["key_len"] is None else s["key_len"]
    return _attention(s["q"], k, v, (j < length[:, None])[:, None])


def _norm_rope(x, w, cos, sin, eps, interleaved):
    x, dt, rot = x.float(), x.dtype, 2 * cos.shape[-1]
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1).to(dt)


def _attention(q, k, v, seen):
    """q [B, Hq, n, d], k and v [B, Hk, L, d], seen [B, n or 1, L]: keys that are not seen have no weight."""
    b, hq, n, d = q.shape
    hk = k.shape[1]
    q5 = q.float().reshape(b, hk, hq // hk, n, d)
    seen = seen[:, None, None]
    x = (q5 @ k.float()[:, :, None].transpose(-1, -2)) * (1 / math.sqrt(d))
    x.masked_fill_(~seen, -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    o = (x @ v.float()[:, :, None]) / x.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.reshape(b, hq, n, d).to(q.dtype)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    d, hq, hk = case["d"], case["Hq"], case["Hk"]
    if case["op"] in ("rope_append", "rope_heads"):
        t = case["T"] if case["op"] == "rope_append" else case["B"] * case["N"]
        heads = hq + hk + (hk if case["op"] == "rope_append" else 0)
        rows = min(t, case["table"]) if case["op"] == "rope_append" else case["N"]
        index = 8 * t if case["op"] == "rope_append" else 0
        return {"bytes": 4 * t * heads * d + 4 * rows * case["rot"] + index, "flops": 8 * t * (hq + hk) * d}
    if case["op"] == "paged":
        nq, kv = _lengths(case)
        pairs = sum(n * m - n * (n - 1) // 2 for n, m in zip(nq, kv))
        table = 4 * sum(-(-m // case["page"]) for m in kv)
        return {"bytes": 4 * sum(nq) * hq * d + 4 * sum(kv) * hk * d + table, "flops": 4 * pairs * hq * d}
    n = _key_lengths(case) if case["ragged"] else [case["Nk"]] * case["B"]
    return {"bytes": 4 * case["B"] * case["Nq"] * hq * d + 4 * sum(n) * hk * d,
            "flops": 4 * case["Nq"] * sum(n) * hq * d}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] in ("rope_append", "rope_heads"):
        c, i = s["cos"].double(), s["sin"].double()
        if case["op"] == "rope_append":
            at = s["positions"].long()
            turn = torch.complex(c[at], i[at])[:, None]
        else:
            turn = torch.complex(c, i)

        def turned(x, w):
            y = x.double().clone()
            if w is not None:
                y = y / (y.pow(2).sum(-1, keepdim=True) / d + s["eps"]).sqrt() * w.double()
            r = case["rot"]
            re, im = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
            z = torch.complex(y[..., re], y[..., im]) * turn
            y[..., re], y[..., im] = z.real, z.imag
            return y

        q, k = turned(s["q"], s["wq"]), turned(s["k"], s["wk"])
        if case["op"] == "rope_heads":
            return {"q": q.contiguous(), "k": k.contiguous()}
        kc, vc = s["k_cache"].double().flatten(0, 1), s["v_cache"].double().flatten(0, 1)
        for n, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                kc[slot], vc[slot] = k[n], s["v"][n].double()
        return {"q": q, "k_cache": kc.view(s["k_cache"].shape), "v_cache": vc.view(s["v_cache"].shape)}
    group = case["Hq"] // case["Hk"]

    def one(q, k, v, first):
        """q [n, d], k and v [m, d]; query i sees the keys up to first + i (all of them where first is None)."""
        out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
        for a in range(0, q.shape[0], 4096):
            x = q[a:a + 4096].double() @ k.double().T / math.sqrt(d)
            if first is not None:
                last = first + a + torch.arange(x.shape[0], device=x.device)
                x[torch.arange(x.shape[1], device=x.device)[None] > last[:, None]] = -math.inf
            out[a:a + 4096] = torch.softmax(x, -1) @ v.double()
        return out

    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "paged":
        nq, kv = _lengths(case)
        at = 0
        for b, (n, m) in enumerate(zip(nq, kv)):
            pages = s["page_table"][b, :-(-m // case["page"])].long()
            for h in range(case["Hk"]):
                k = s["k_cache"][pages, :, h].flatten(0, 1)[:m]
                v = s["v_cache"][pages, :, h].flatten(0, 1)[:m]
                for e in range(h * group, (h + 1) * group):
                    out[at:at + n, e] = one(s["q"][at:at + n, e], k, v, m - n)
            at += n
        return out
    n = _key_lengths(case) if case["ragged"] else [case["Nk"]] * case["B"]
    for b in range(case["B"]):
        for e in range(case["Hq"]):
            h = e // group
            out[b, e] = one(s["q"][b, e], s["k"][b, h, :n[b]], s["v"][b, h, :n[b]], None)
    return out
