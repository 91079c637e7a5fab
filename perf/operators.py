"""Workloads of the verify-step operators around the windowed attention, with
their plain forms.

  sink    swa_sink_verify_attn: sliding-window attention in which the first
          few tokens stay visible, on a contiguous or paged cache, optionally
          writing the block's new K/V rows into it
  rope    swa_qk_norm_rope / swa_qk_norm_rope_append: RMS norm of every query
          and key head and the position rotation in one pass, the K/V rows
          returned or written straight into the cache
  sample  swa_sample_accept: a token per verify row from given random numbers
          under temperature, top-k, top-p and min-p, and the accepted prefix

A case is a dict of plain values.  ``prepare`` draws its inputs on the GPU,
``run`` makes one pass (plain torch while ``own`` is false, the library's
calls when it is true), ``work`` counts what a pass cannot do without and
``exact`` evaluates the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

_BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases

def _sink(name, B, q, Hq, Hkv, D, W, S, ctx, L, page=0, append=False, lens=0):
    return {"name": name, "op": "sink", "B": B, "q": q, "Hq": Hq, "Hkv": Hkv, "D": D, "W": W,
            "S": S, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "L": L, "page": page, "append": append,
            "lens": lens}


def _rope(name, B, q, Hq, Hkv, D, rot, interleaved, norm, ctx, L=0, page=0, lens=0):
    """L = 0: the rows are returned; L > 0: written into a cache of L rows."""
    return {"name": name, "op": "rope", "B": B, "q": q, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
            "interleaved": interleaved, "norm": norm, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "L": L,
            "page": page, "lens": lens}


def _sample(name, B, q, V, mode, keep=False, masked=False):
    return {"name": name, "op": "sample", "B": B, "q": q, "V": V, "mode": mode, "keep": keep,
            "masked": masked}


def listed():
    return [
        # one conversation's verify block (1 committed + 7 drafted tokens): latency
        _sink("sink_single_q8", 1, 8, 8, 2, 256, 188, 4, (4096, 4096), 4096),
        # a served batch on a paged cache, the block's K/V rows written by the call
        _sink("sink_paged_append_b64_q8", 64, 8, 8, 2, 256, 188, 4, (200, 4096), 4096, page=16,
              append=True),
        # the bandwidth-bound batch: long windows, hundreds of sequences
        _sink("sink_stress_b512_w1024_q8", 512, 8, 8, 2, 256, 1024, 4, (1100, 4096), 4096),
        # prefill chunks under a small window with a longer pinned prefix
        _sink("sink_prefill_b8_q512_d128", 8, 512, 8, 2, 128, 600, 67, (900, 2048), 2048, page=64),
        # single-token decode at the small head size, odd window and prefix
        _sink("sink_decode_b33_q1_d64", 33, 1, 8, 4, 64, 333, 5, (40, 1000), 1000),
        # the verify block of one conversation, rows handed to the attention call
        _rope("rope_single_q8", 1, 8, 8, 2, 256, 256, False, True, (4096, 4096)),
        # a served batch, K/V rows written straight into the pages
        _rope("rope_paged_append_b64_q8", 64, 8, 8, 2, 256, 256, False, True, (200, 4096),
              L=4096, page=16),
        # long draft blocks of the stress batch at positions far into the context
        _rope("rope_stress_b512_q64", 512, 64, 8, 2, 256, 128, False, True, (1024, 32768)),
        # one conversation's verify block over a 262,144-token vocabulary: latency
        _sample("sample_single_q8", 1, 8, 262144, "topk_topp"),
        # a served batch whose requests each bring their own settings
        _sample("sample_mixed_b64_q8", 64, 8, 262144, "mixed"),
        # no filter at all: every logit counts
        _sample("sample_plain_b64_q1", 64, 1, 262144, "plain"),
        # a pruned head (keep set) whose grammar masks columns, min-p
        _sample("sample_keep_b48_q5", 48, 5, 12001, "min_p", keep=True, masked=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sink", "rope", "sample"])
    while True:
        if op == "sink":
            D, Hkv, G = rng.choice([64, 128, 256]), rng.choice([1, 2, 3, 4]), rng.choice([1, 2, 4, 8])
            q, B = _log(rng, 1, 512), _log(rng, 1, 512)
            W, S = _log(rng, 1, 2048), rng.choice([0, rng.randint(1, 8), rng.randint(1, 128)])
            page = rng.choice([0, 0, 8, 16, 24, 64])
            L = _log(rng, max(64, q), 4096)
            L = L if page == 0 else -(-L // page) * page
            c = _sink("", B, q, G * Hkv, Hkv, D, W, S, (q, L), L, page, rng.random() < 0.4,
                      rng.randint(1, 10 ** 6))
            w = work(c)
            if (B * Hkv * L * D <= 512 * 2 * 4096 * 256 // 4 and w["flops"] <= 2e10 and
                    w["bytes"] <= 1.0e9 and B * Hkv * G * q * min(L, W + q + S) <= 1 << 27):
                break
        elif op == "rope":
            D, Hkv, G = rng.choice([64, 128, 256]), rng.choice([1, 2, 3, 4]), rng.choice([1, 2, 4, 8])
            q, B = _log(rng, 1, 512), _log(rng, 1, 512)
            rot = rng.choice([D, D, D // 2, D // 4])
            page = rng.choice([0, 16, 64])
            L = rng.choice([0, _log(rng, max(64, q), 4096)])
            L = L if page == 0 else -(-L // page) * page
            if L == 0:
                page = 0
            hi = L if L > 0 else rng.choice([4096, 32768, 1000000])
            c = _rope("", B, q, G * Hkv, Hkv, D, rot, rng.random() < 0.4, rng.random() < 0.8,
                      (q, max(q, hi)), L, page, rng.randint(1, 10 ** 6))
            if work(c)["bytes"] <= 4.0e8 and B * Hkv * max(L, 1) * D <= 512 * 2 * 4096 * 256 // 4:
                break
        else:
            V, q, B = _log(rng, 200, 262144), _log(rng, 1, 64), _log(rng, 1, 256)
            c = _sample("", B, q, V, rng.choice(["topk_topp", "nucleus", "plain", "min_p", "mixed"]),
                        rng.random() < 0.3, rng.random() < 0.3)
            if B * q * V <= 64 * 8 * 262144:
                break
    del c["name"]
    return c


# ------------------------------------------------------------------ work

def _lens(case):
    rng = random.Random(case["lens"])
    return [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]


def work(case):
    if case["op"] == "sink":
        q, Hq, Hkv, D, W, S = (case[k] for k in ("q", "Hq", "Hkv", "D", "W", "S"))
        keys = pairs = 0
        for n in _lens(case):
            p0 = n - q
            lo = max(0, p0 - W + 1)
            keys += n - lo + min(S, lo)
            for i in range(q):
                l = max(0, p0 + i - W + 1)
                pairs += p0 + i + 1 - l + min(S, l)
        rows = case["B"] * q * Hq
        kv = keys * Hkv * D * 2 * 2
        if case["append"]:
            kv += case["B"] * q * Hkv * D * 2 * 2      # the new rows are read and stored
        return {"bytes": kv + rows * (D * 2 * 2 + 4) + case["B"] * 8, "flops": pairs * Hq * D * 4}
    if case["op"] == "rope":
        heads = case["B"] * case["q"] * (case["Hq"] + 2 * case["Hkv"])
        return {"bytes": heads * case["D"] * 2 * 2 + case["rot"] * 2 + 2 * case["D"] * 4,
                "flops": heads * case["D"] * 6}
    n = case["B"] * case["q"] * case["V"]
    return {"bytes": n * 2 + case["B"] * case["q"] * 16 + (case["V"] * 4 if case["keep"] else 0),
            "flops": n * 3}


# --------------------------------------------------------------- prepare

def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=_BF16)


def _cache(case, gen):
    """K and V caches, and the block table of a shuffled pool if paged."""
    B, Hkv, D, L, page = case["B"], case["Hkv"], case["D"], case["L"], case["page"]
    if page == 0:
        return _randn((B, Hkv, L, D), gen), _randn((B, Hkv, L, D), gen), None
    nb = L // page
    num = B * nb + 3
    table = torch.randperm(num, generator=gen, device="cuda")[:B * nb].view(B, nb)
    return (_randn((num, Hkv, page, D), gen), _randn((num, Hkv, page, D), gen),
            table.to(torch.int32).contiguous())


def _outliers(k, gen):
    """1% of the entries times 8, in place and by slices."""
    flat = k.view(-1)
    for part in flat.split(1 << 26):
        part[torch.rand(part.shape, generator=gen, device="cuda") < 0.01] *= 8


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "sample":
        _prepare_sample(case, st, gen)
        return st
    lens = _lens(case)
    st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["q_pos"] = st["seq_lens"] - case["q"]
    B, q, Hq, Hkv, D = (case[k] for k in ("B", "q", "Hq", "Hkv", "D"))
    if case["op"] == "sink":
        st["q"] = _randn((B, q, Hq, D), gen)
        st["k_cache"], st["v_cache"], st["table"] = _cache(case, gen)
        _outliers(st["k_cache"], gen)
        if case["append"]:
            st["k_new"], st["v_new"] = _randn((B, q, Hkv, D), gen), _randn((B, q, Hkv, D), gen)
        return st
    # the fused projection's output: all query heads, then key, then value heads
    qkv = _randn((B, q, Hq + 2 * Hkv, D), gen) * (0.5 + 3 * torch.rand(
        (1, 1, Hq + 2 * Hkv, 1), generator=gen, device="cuda"))
    qkv = qkv.to(_BF16)
    st["q"], st["k"], st["v"] = qkv.split([Hq, Hkv, Hkv], dim=2)
    st["qw"] = st["kw"] = None
    if case["norm"]:
        st["qw"] = 0.5 + torch.rand(D, generator=gen, device="cuda")
        st["kw"] = 0.5 + torch.rand(D, generator=gen, device="cuda")
    i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
    st["inv_freq"] = (10000.0 ** (-2 * i / case["rot"])).float()
    st["eps"] = 1e-6
    if case["L"]:
        st["k_cache"], st["v_cache"], st["table"] = _cache(case, gen)
    return st


def _prepare_sample(case, st, gen):
    B, q, V = case["B"], case["q"], case["V"]
    x = _randn((B, q, V), gen) * 2
    # a few likely tokens above the bulk
    n = min(16, V)
    cols = torch.randint(0, V, (B, q, n), generator=gen, device="cuda")
    x.scatter_(2, cols, (5 + 9 * torch.rand((B, q, n), generator=gen, device="cuda")).to(_BF16))
    if case["masked"]:
        for b in range(B):
            x[b].masked_fill_(torch.rand((q, V), generator=gen, device="cuda") < 0.25,
                              float("-inf"))
    st["logits"] = x
    st["u"] = torch.rand((B, q), generator=gen, device="cuda")
    st["keep"] = (torch.randperm(4 * V, generator=gen, device="cuda")[:V].to(torch.int32)
                  if case["keep"] else None)
    st["draft"] = None
    if q > 1:
        top = x[:, :-1].argmax(dim=2)
        rnd = torch.randint(0, V, (B, q - 1), generator=gen, device="cuda")
        col = torch.where(torch.rand((B, q - 1), generator=gen, device="cuda") < 0.8, top, rnd)
        st["draft"] = (st["keep"][col] if case["keep"] else col).to(torch.int32).contiguous()

    def full(v, dtype=torch.float32):
        return torch.full((B,), v, dtype=dtype, device="cuda")

    def pick(values, dtype=torch.float32):
        i = torch.randint(0, len(values), (B,), generator=gen, device="cuda")
        return torch.tensor(values, dtype=dtype, device="cuda")[i]

    st["top_k"] = st["top_p"] = st["min_p"] = None
    mode = case["mode"]
    if mode == "mixed":
        st["temperature"] = pick([0.0, 0.6, 0.8, 1.0, 1.3])
        st["top_k"] = pick([0, 0, 20, 64, 1000], torch.int32)
        st["top_p"] = pick([0.8, 0.95, 1.0, 1.0])
        st["min_p"] = pick([0.0, 0.0, 0.02, 0.1])
    elif mode == "topk_topp":
        st["temperature"], st["top_k"], st["top_p"] = full(0.8), full(50, torch.int32), full(0.95)
    elif mode == "nucleus":
        st["temperature"], st["top_p"] = full(1.0), full(0.9)
    elif mode == "min_p":
        st["temperature"], st["min_p"] = full(1.2), full(0.05)
    else:
        st["temperature"] = full(1.0)


# ------------------------------------------------------------------- run

def run(st):
    op = st["case"]["op"]
    if own:
        return {"sink": _own_sink, "rope": _own_rope, "sample": _own_sample}[op](st)
    return {"sink": _plain_sink, "rope": _plain_rope, "sample": _plain_sample}[op](st)


def _call(st, name, *args, **kw):
    """The library call, validated and marshalled once and then re-issued, as
    a serving loop does."""
    if "call" not in st:
        import sliding_window_speculative_gb300 as swa
        st["call"] = swa.prepare(getattr(swa, name), *args, **kw)
    return st["call"]()


def _own_sink(st):
    c = st["case"]
    out, lse = _call(st, "swa_sink_verify_attn", st["q"], st["k_cache"], st["v_cache"],
                     st["seq_lens"], st["q_pos"], c["W"], c["S"], c["D"] ** -0.5,
                     k_new=st.get("k_new"), v_new=st.get("v_new"), block_table=st["table"])
    return (out, lse, st["k_cache"], st["v_cache"]) if c["append"] else (out, lse)


def _own_rope(st):
    c = st["case"]
    if c["L"]:
        q = _call(st, "swa_qk_norm_rope_append", st["q"], st["k"], st["v"], st["qw"], st["kw"],
                  st["eps"], st["inv_freq"], st["k_cache"], st["v_cache"], st["seq_lens"],
                  st["q_pos"], interleaved=c["interleaved"], block_table=st["table"])
        return q, st["k_cache"], st["v_cache"]
    return _call(st, "swa_qk_norm_rope", st["q"], st["k"], st["v"], st["qw"], st["kw"], st["eps"],
                 st["inv_freq"], st["q_pos"], interleaved=c["interleaved"])


def _own_sample(st):
    return _call(st, "swa_sample_accept", st["logits"], st["u"], st["temperature"],
                 top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"], draft=st["draft"],
                 keep_ids=st["keep"])


def _rows(case, st, cache, b, j):
    """Cache rows [..., Hkv, D] of positions j of sequences b (index arrays)."""
    if case["page"] == 0:
        return cache[b, :, j]
    page = st["table"].long()[b, j // case["page"]]
    return cache[page, :, j % case["page"]]


def _write_rows(case, st, cache, rows):
    """Rows [B, q, Hkv, D] into the cache at positions q_pos + i."""
    B, q = rows.shape[:2]
    b = torch.arange(B, device="cuda")[:, None].expand(B, q)
    j = st["q_pos"].long()[:, None] + torch.arange(q, device="cuda")
    if case["page"] == 0:
        cache[b, :, j] = rows
    else:
        cache[st["table"].long()[b, j // case["page"]], :, j % case["page"]] = rows


def _plain_sink(st):
    c = st["case"]
    B, q, Hq, Hkv, D, W, S, L = (c[k] for k in ("B", "q", "Hq", "Hkv", "D", "W", "S", "L"))
    if c["append"]:
        _write_rows(c, st, st["k_cache"], st["k_new"])
        _write_rows(c, st, st["v_cache"], st["v_new"])
    G = Hq // Hkv
    qp, sl = st["q_pos"].long(), st["seq_lens"].long()
    lo = (qp - W + 1).clamp_min(0)
    sinks = torch.arange(min(S, L), device="cuda").expand(B, -1)
    win = lo[:, None] + torch.arange(min(L, W + q - 1), device="cuda")
    # a position that both parts list counts in the window part only
    j = torch.cat([sinks, win], dim=1)
    once = torch.cat([sinks < lo[:, None], win < sl.clamp_max(L)[:, None]], dim=1)
    p = qp[:, None] + torch.arange(q, device="cuda")
    jj, pp = j[:, None, :], p[:, :, None]
    vis = once[:, None, :] & (jj <= pp) & ((jj > pp - W) | (jj < S))      # [B, q, n]
    jc = j.clamp(0, L - 1)
    b = torch.arange(B, device="cuda")[:, None].expand_as(jc)
    k = _rows(c, st, st["k_cache"], b, jc).float().permute(0, 2, 1, 3)    # [B, Hkv, n, D]
    qf = st["q"].float().view(B, q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, q * G, D)
    s = torch.matmul(qf, k.transpose(2, 3)).view(B, Hkv, q, G, -1) * D ** -0.5
    s = torch.where(vis[:, None, :, None, :], s, float("-inf"))
    m = s.amax(dim=-1, keepdim=True)
    e = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
    l = e.sum(dim=-1, keepdim=True)
    v = _rows(c, st, st["v_cache"], b, jc).float().permute(0, 2, 1, 3)
    o = torch.matmul(e.view(B, Hkv, q * G, -1), v).view(B, Hkv, q, G, D)
    o = torch.where(l > 0, o / l, 0.0)
    lse = (m + torch.log(l)).squeeze(-1)
    out = o.permute(0, 2, 1, 3, 4).reshape(B, q, Hq, D).to(_BF16)
    lse = lse.permute(0, 2, 1, 3).reshape(B, q, Hq)
    return (out, lse, st["k_cache"], st["v_cache"]) if c["append"] else (out, lse)


def _plain_rope(st):
    c = st["case"]
    p = st["q_pos"].double()[:, None] + torch.arange(c["q"], dtype=torch.float64, device="cuda")
    ang = p[:, :, None, None] * st["inv_freq"].double()                    # [B, q, 1, rot/2]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()

    def turn(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + st["eps"]) * w
        rot = c["rot"]
        r, rest = x[..., :rot], x[..., rot:]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        return torch.cat([r, rest], dim=-1).to(_BF16)

    q, k = turn(st["q"], st["qw"]), turn(st["k"], st["kw"])
    if c["L"]:
        _write_rows(c, st, st["k_cache"], k)
        _write_rows(c, st, st["v_cache"], st["v"])
        return q, st["k_cache"], st["v_cache"]
    return q, k, st["v"].contiguous()


def _plain_sample(st):
    c = st["case"]
    B, q, V = c["B"], c["q"], c["V"]
    step = max(1, (1 << 25) // (q * V))     # sequences at a time, for the sorted copies' memory
    toks, lps = [], []
    for b0 in range(0, B, step):
        sl = slice(b0, min(B, b0 + step))
        x = st["logits"][sl].float()
        x = torch.where(torch.isnan(x), float("-inf"), x) + 0.0      # (-0 is 0)
        vals, idx = torch.sort(x, dim=2, descending=True, stable=True)
        top = vals[..., :1].double()
        t = st["temperature"][sl].double()[:, None, None]
        w = torch.exp((vals.double() - top) / torch.where(t > 0, t, 1.0))
        w = torch.where(torch.isinf(top), (vals == top).double(), w)
        first = torch.arange(V, device="cuda") == 0
        keep = ((t > 0) & (vals > float("-inf"))) | first
        if st["top_k"] is not None:
            k = st["top_k"][sl].long()[:, None, None]
            keep = keep & ((k <= 0) | (torch.arange(V, device="cuda") < k))
        if st["top_p"] is not None:
            tp = st["top_p"][sl].double()[:, None, None]
            cum = torch.cumsum(torch.where(keep, w, 0.0), dim=2)
            before = torch.cat([torch.zeros_like(cum[..., :1]), cum[..., :-1]], dim=2)
            keep = keep & ((tp >= 1) | (before < tp * cum[..., -1:]))
        if st["min_p"] is not None:
            keep = keep & (w >= st["min_p"][sl].double()[:, None, None])
        keep = keep | first
        cum = torch.cumsum(torch.where(keep, w, 0.0), dim=2)
        total = cum[..., -1:]
        n = keep.sum(dim=2, keepdim=True)
        m = (cum <= st["u"][sl].double()[:, :, None] * total).sum(dim=2, keepdim=True)
        m = torch.minimum(m, n - 1)
        col = torch.gather(idx, 2, m).squeeze(2)
        lps.append(torch.log(torch.gather(w, 2, m) / total).squeeze(2).float())
        toks.append((st["keep"][col] if st["keep"] is not None else col).to(torch.int32))
    tokens, logprobs = torch.cat(toks), torch.cat(lps)
    if st["draft"] is None:
        accepted = torch.zeros((B,), dtype=torch.int32, device="cuda")
    else:
        same = (tokens[:, :-1] == st["draft"]).to(torch.int32)
        accepted = torch.cumprod(same, dim=1).sum(dim=1).to(torch.int32)
    return tokens, accepted, logprobs


# ----------------------------------------------------------------- exact

def exact(case, seed):
    st = prepare(case, seed)
    return {"sink": _exact_sink, "rope": _exact_rope, "sample": _exact_sample}[case["op"]](case, st)


def _position_view(case, st, cache, b, js):
    """[n, Hkv, D] rows of sequence b at the listed positions."""
    if case["page"] == 0:
        return cache[b][:, js].transpose(0, 1)
    pages = st["table"][b].long()
    return cache[pages[js // case["page"]], :, js % case["page"]]


def _put(case, st, cache, rows):
    for b, n in enumerate(_lens(case)):
        for i in range(case["q"]):
            j = n - case["q"] + i
            if case["page"] == 0:
                cache[b, :, j] = rows[b, i]
            else:
                cache[int(st["host_table"][b, j // case["page"]]), :, j % case["page"]] = rows[b, i]


def _exact_sink(case, st):
    q, Hq, Hkv, D, W, S, L = (case[k] for k in ("q", "Hq", "Hkv", "D", "W", "S", "L"))
    if case["B"] * q > 20000:
        return None
    if case["append"]:
        st["host_table"] = None if st["table"] is None else st["table"].cpu().numpy()
        _put(case, st, st["k_cache"], st["k_new"])
        _put(case, st, st["v_cache"], st["v_new"])
    out = torch.zeros((case["B"], q, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], q, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        p0 = n - q
        js = sorted(set(range(min(S, n))) | set(range(max(0, p0 - W + 1), n)))
        js = torch.tensor(js, device="cuda")
        k = _position_view(case, st, st["k_cache"], b, js).double()
        v = _position_view(case, st, st["v_cache"], b, js).double()
        p = torch.arange(p0, n, device="cuda")[:, None]
        hidden = (js > p) | ((js <= p - W) & (js >= S))
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            s = torch.einsum("ihd,nd->ihn", st["q"][b, :, heads].double(), k[:, h]) / math.sqrt(D)
            s = s.masked_fill(hidden[:, None, :], float("-inf"))
            z = torch.logsumexp(s, dim=-1)
            lse[b, :, heads] = z
            out[b, :, heads] = torch.einsum("ihn,nd->ihd", torch.exp(s - z[..., None]), v[:, h])
    if case["append"]:
        return out, lse, st["k_cache"], st["v_cache"]
    return out, lse


def _exact_rope(case, st):
    B, n, rot = case["B"], case["q"], case["rot"]
    pos = torch.tensor([[l - n + i for i in range(n)] for l in _lens(case)], dtype=torch.float64,
                       device="cuda")
    turn = torch.polar(torch.ones((B, n, rot // 2), dtype=torch.float64, device="cuda"),
                       pos[..., None] * st["inv_freq"].double())

    def heads(x, w):
        out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for h in range(x.shape[2]):
            y = x[:, :, h].double()
            if w is not None:
                y = y / torch.sqrt(y.square().sum(dim=-1, keepdim=True) / case["D"] + st["eps"])
                y = y * w.double()
            if case["interleaved"]:
                z = torch.view_as_complex(y[..., :rot].reshape(B, n, rot // 2, 2).contiguous())
                y[..., :rot] = torch.view_as_real(z * turn).reshape(B, n, rot)
            else:
                z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
                y = torch.cat([z.real, z.imag, y[..., rot:]], dim=-1)
            out[:, :, h] = y
        return out

    q, k = heads(st["q"], st["qw"]), heads(st["k"], st["kw"])
    if case["L"] == 0:
        return q, k, st["v"].double()
    if B * n > 20000:
        return q, None, None
    st["host_table"] = None if st["table"] is None else st["table"].cpu().numpy()
    kc = st["k_cache"].double()
    _put(case, st, kc, k)
    _put(case, st, st["v_cache"], st["v"])
    return q, kc, st["v_cache"]


def _exact_sample(case, st):
    """By counting: columns with the same 16 bits have the same weight, so a
    row is its distinct values in falling order and how often each occurs."""
    B, q, V = case["B"], case["q"], case["V"]
    if B * q * V > 64 * 8 * 262144 or B * q > 8192:
        return None
    bits = st["logits"].view(torch.int16).cpu().numpy().view(np.uint16)
    of_bits = (np.arange(65536, dtype=np.uint32) << 16).view(np.float32)
    host = {k: None if st[k] is None else st[k].cpu().numpy()
            for k in ("u", "temperature", "top_k", "top_p", "min_p", "keep", "draft")}
    tokens = np.zeros((B, q), dtype=np.int32)
    logprobs = np.zeros((B, q))
    accepted = np.zeros(B, dtype=np.int32)
    for b in range(B):
        T = float(host["temperature"][b])
        for i in range(q):
            row = bits[b, i]
            row = np.where(row == 0x8000, 0, row).astype(np.uint16)      # -0 is 0
            count = np.bincount(row, minlength=65536)
            here = np.flatnonzero(count)
            here = here[of_bits[here] > -np.inf]                          # neither NaN nor -inf
            if here.size == 0:
                col, lp = 0, 0.0
            else:
                here = here[np.argsort(-of_bits[here].astype(np.float64), kind="stable")]
                val, cnt = of_bits[here].astype(np.float64), count[here]
                col, lp = _pick(val, cnt, T, {k: host[k][b] if host[k] is not None else None
                                              for k in ("top_k", "top_p", "min_p")},
                                float(host["u"][b, i]),
                                lambda n, r: int(np.flatnonzero(row == here[n])[r]))
            tokens[b, i] = host["keep"][col] if host["keep"] is not None else col
            logprobs[b, i] = lp
        while accepted[b] < q - 1 and tokens[b, accepted[b]] == host["draft"][b, accepted[b]]:
            accepted[b] += 1
    dev = "cuda"
    return (torch.from_numpy(tokens).to(dev), torch.from_numpy(accepted).to(dev),
            torch.from_numpy(logprobs).to(dev))


def _pick(val, cnt, T, f, u, column):
    if not T > 0:
        return column(0, 0), 0.0
    w = (val == val[0]).astype(np.float64) if np.isinf(val[0]) else np.exp((val - val[0]) / T)
    left = cnt.astype(np.int64)
    if f["top_k"] is not None and f["top_k"] > 0:
        left = np.minimum(left, np.maximum(0, int(f["top_k"]) - (np.cumsum(left) - left)))
    if f["top_p"] is not None and f["top_p"] < 1:
        mass = left * w
        need = float(f["top_p"]) * mass.sum() - (np.cumsum(mass) - mass)
        # copies of a value kept while the mass before them is short of the target
        more = np.ceil(np.maximum(need, 0) / np.maximum(w, 1e-300))
        left = np.minimum(left, np.minimum(more, 1 << 40).astype(np.int64))
    if f["min_p"] is not None:
        left = np.where(w >= float(f["min_p"]), left, 0)
    left[0] = max(left[0], 1)
    mass = left * w
    cum, total = np.cumsum(mass), mass.sum()
    n = min(int(np.searchsorted(cum, u * total, side="right")), int(np.flatnonzero(left)[-1]))
    r = int((u * total - (cum[n] - mass[n])) / w[n])
    return column(n, min(max(r, 0), int(left[n]) - 1)), math.log(w[n] / total)
