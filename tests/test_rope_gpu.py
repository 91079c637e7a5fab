"""GPU parity of the head norm + rotation against its fp64 definition.

Tolerance, derived: the result is rounded to bf16 once (half a step: 2^-8 of
the value).  Before that, in fp32: the mean of D <= 256 squares (a lane adds
16 in order, the lanes by a tree of at most 4 steps: < 20 roundings, halved by
the root), the root's 2 units, two products: below 2^-19 of the value; the
angle is off by at most 2^-25 turns (2^-22 rad) and cosine and sine by 2
units, so a rotated value by less than 2^-20 (|a| + |b|).  Together
2^-8 |y| + 2^-18 (|a| + |b|)."""
import numpy as np
import pytest
import torch

import oracle.verify_step as vs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


def _f64(t):
    return t.to(torch.float64).cpu().numpy()


def _case(B, q_len, Hq, Hkv, D, rot, seed, pos=None, q_norm=True, k_norm=True, packed=True):
    g = torch.Generator().manual_seed(seed)
    H = Hq + 2 * Hkv
    x = torch.randn((B, q_len, H, D), generator=g) * torch.logspace(-2, 2, H)[:, None]
    x = x.to(torch.bfloat16).cuda()
    parts = x.split([Hq, Hkv, Hkv], dim=2)
    if not packed:
        parts = [p.contiguous() for p in parts]
    w = [(0.5 + torch.rand(D, generator=g)).cuda() for _ in range(2)]
    f = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(rot, 1))).float().cuda()
    if pos is None:
        pos = torch.randint(0, 5000, (B,), generator=g).tolist()
    return dict(q=parts[0], k=parts[1], v=parts[2], q_weight=w[0] if q_norm else None,
                k_weight=w[1] if k_norm else None, eps=1e-6, inv_freq=f if rot else None,
                q_pos=torch.tensor(pos, dtype=torch.int32).cuda())


def _want(c, name, interleaved):
    x, w = c[name], c[name + "_weight"]
    B, q_len, H, D = x.shape
    pos = (c["q_pos"].cpu().numpy()[:, None].astype(np.int64) + np.arange(q_len)).reshape(-1)
    y, size = vs.norm_rope(_f64(x).reshape(B * q_len, H, D), None if w is None else _f64(w), c["eps"],
                           None if c["inv_freq"] is None else _f64(c["inv_freq"]), pos, interleaved)
    return y.reshape(x.shape), size.reshape(x.shape)


def _close(got, want, size, slack=0.0):
    err = np.abs(_f64(got) - want)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -18 + slack) * size
    assert np.all(err <= tol), (err - tol).max()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,q_len,Hq,Hkv,D,rot", [
    (1, 8, 8, 2, 256, 256), (3, 5, 4, 1, 128, 128), (2, 1, 9, 3, 64, 64), (5, 7, 8, 8, 64, 16),
    (2, 512, 2, 1, 128, 32), (1, 1, 1, 1, 256, 48), (40, 64, 8, 2, 256, 128), (7, 3, 6, 2, 128, 0),
    (300, 33, 3, 3, 64, 48),
])
def test_matches_definition(B, q_len, Hq, Hkv, D, rot, interleaved):
    import sliding_window_speculative_gb300 as swa
    c = _case(B, q_len, Hq, Hkv, D, rot, seed=B + q_len + D)
    q, k, v = swa.swa_qk_norm_rope(**c, interleaved=interleaved)
    torch.cuda.synchronize()
    _close(q, *_want(c, "q", interleaved))
    _close(k, *_want(c, "k", interleaved))
    assert torch.equal(v, c["v"])


@pytest.mark.parametrize("q_norm,k_norm,packed", [(True, False, True), (False, True, False),
                                                  (False, False, True)])
def test_norms_are_optional(q_norm, k_norm, packed):
    import sliding_window_speculative_gb300 as swa
    c = _case(2, 9, 8, 2, 128, 128, seed=3, q_norm=q_norm, k_norm=k_norm, packed=packed)
    q, k, v = swa.swa_qk_norm_rope(**c)
    torch.cuda.synchronize()
    _close(q, *_want(c, "q", False))
    _close(k, *_want(c, "k", False))
    assert torch.equal(v, c["v"])
    c["inv_freq"] = None
    q, k, v = swa.swa_qk_norm_rope(**c)
    torch.cuda.synchronize()
    if not q_norm:
        assert torch.equal(q, c["q"])      # nothing to do: the same bits
    if not k_norm:
        assert torch.equal(k, c["k"])


@pytest.mark.parametrize("pos", [0, 1, 65535, 1 << 20, (1 << 24) + 1, (1 << 31) - 9, (1 << 31) - 1])
def test_far_positions(pos):
    """The angle keeps its fraction of a turn at any position: 2^-53 of the
    fp64 angle (the definition's own rounding) is the only added slack."""
    import sliding_window_speculative_gb300 as swa
    c = _case(2, 8, 4, 2, 256, 256, seed=5, pos=[pos, pos // 3])
    q, k, _ = swa.swa_qk_norm_rope(**c)
    torch.cuda.synchronize()
    slack = 2.0 ** -52 * (pos + 8)
    _close(q, *_want(c, "q", False), slack=slack)
    _close(k, *_want(c, "k", False), slack=slack)


@pytest.mark.parametrize("scale", [1.0, -1.0, 7.5, 1e-20, 3.0e5, 0.0])
def test_any_frequency(scale):
    """Frequencies of any size and sign: large ones by whole turns, 0 and
    vanishing ones leave the row as it is."""
    import sliding_window_speculative_gb300 as swa
    c = _case(3, 4, 4, 2, 64, 64, seed=6, pos=[0, 17, 900])
    c["inv_freq"] = c["inv_freq"] * scale
    q, _, _ = swa.swa_qk_norm_rope(**c)
    torch.cuda.synchronize()
    _close(q, *_want(c, "q", False), slack=2.0 ** -52 * 1000 * abs(scale))


def test_zero_rows_and_nan_stay_in_their_row():
    import sliding_window_speculative_gb300 as swa
    c = _case(2, 3, 4, 2, 128, 128, seed=8)
    base = swa.swa_qk_norm_rope(**c)[0].clone()
    x = c["q"].clone()
    x[0, 1, 2] = 0
    x[1, 2, 3, 5] = float("nan")
    c["q"] = x
    q = swa.swa_qk_norm_rope(**c)[0]
    torch.cuda.synchronize()
    assert torch.all(q[0, 1, 2] == 0)
    assert torch.all(torch.isnan(q[1, 2, 3]))
    same = torch.ones(q.shape[:3], dtype=torch.bool, device="cuda")
    same[0, 1, 2] = same[1, 2, 3] = False
    assert torch.equal(q[same], base[same])


def _caches(c, L, page, seed=1):
    B, Hkv, D = c["q"].shape[0], c["k"].shape[2], c["q"].shape[3]
    g = torch.Generator(device="cuda").manual_seed(seed)
    if page == 0:
        shape, table = (B, Hkv, L, D), None
    else:
        nb = L // page
        shape = (B * nb + 3, Hkv, page, D)
        table = torch.randperm(B * nb + 3, generator=g, device="cuda")[:B * nb].view(B, nb)
        table = table.to(torch.int32).contiguous()
    return [torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)], table


@pytest.mark.parametrize("page", [0, 8, 24, 64])
@pytest.mark.parametrize("D,q_len", [(256, 8), (64, 1), (128, 70)])
def test_append_writes_its_rows_and_nothing_else(page, D, q_len):
    import sliding_window_speculative_gb300 as swa
    L = 192
    # one block inside the cache, one ending at seq_len < its end (rows past it
    # dropped), one that runs over the cache's end, one at position 0
    pos, lens = [33, 20, L - q_len // 2, 0], [33 + q_len, 20 + q_len // 2, L, q_len]
    c = _case(4, q_len, 4, 2, D, D, seed=9, pos=pos)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    (kc, vc), table = _caches(c, L, page)
    k0, v0 = kc.clone(), vc.clone()
    q_ref, k_new, v_new = swa.swa_qk_norm_rope(**c)
    q = swa.swa_qk_norm_rope_append(**c, k_cache=kc, v_cache=vc, seq_lens=sl, block_table=table)
    torch.cuda.synchronize()
    assert torch.equal(q, q_ref)
    for b in range(4):
        for i in range(q_len):
            j = pos[b] + i
            if j >= min(lens[b], L):
                continue
            if page == 0:
                k0[b, :, j], v0[b, :, j] = k_new[b, i], v_new[b, i]
            else:
                p = int(table[b, j // page])
                k0[p, :, j % page], v0[p, :, j % page] = k_new[b, i], v_new[b, i]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_two_streams_prepared_and_captured():
    """Two overlapping calls on streams of their own (the operator keeps no
    state), a prepared call on new contents, and a captured graph replayed."""
    import sliding_window_speculative_gb300 as swa
    cs = [_case(64, 8, 8, 2, 256, 256, seed=s) for s in (1, 2)]
    want = [[t.clone() for t in swa.swa_qk_norm_rope(**c)] for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [swa.swa_qk_norm_rope(**c, stream=s) for c, s in zip(cs, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))
    call = swa.prepare(swa.swa_qk_norm_rope, **cs[0])
    graph = torch.cuda.CUDAGraph()
    outs = [torch.empty_like(t) for t in want[0]]
    with torch.cuda.graph(graph):
        swa.swa_qk_norm_rope(**cs[0], q_out=outs[0], k_out=outs[1], v_out=outs[2])
    qkv = torch.cat([cs[1][n] for n in "qkv"], dim=2)
    for n, part in zip("qkv", qkv.split([8, 2, 2], dim=2)):
        cs[0][n].copy_(part)
    for n in ("q_weight", "k_weight", "q_pos"):
        cs[0][n].copy_(cs[1][n])
    got = call()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    assert all(torch.equal(a, b) for a, b in zip(outs, want[1]))


def test_binding_refuses_uneven_strides():
    import sliding_window_speculative_gb300 as swa
    c = _case(4, 6, 8, 2, 128, 128, seed=4)
    for bad in (c["q"].transpose(1, 2).contiguous().transpose(1, 2), c["q"][:, :3],
                c["q"][..., ::2]):
        with pytest.raises(ValueError):
            swa.swa_qk_norm_rope(**{**c, "q": bad, "k": c["k"][:, :bad.shape[1]],
                                    "v": c["v"][:, :bad.shape[1]]})
    # every other token of the whole batch is evenly spaced: taken as it is
    e = {n: c[n][:, ::2] for n in "qkv"}
    got = swa.swa_qk_norm_rope(**{**c, **e})
    ref = swa.swa_qk_norm_rope(**{**c, **{n: t.contiguous() for n, t in e.items()}})
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_offsets_past_32_bits():
    """Rows written past element 2^31 of a cache, and inputs whose token
    stride takes them there."""
    import sliding_window_speculative_gb300 as swa
    D, n = 256, 4
    L = (1 << 31) // D + 1024
    c = _case(1, n, 2, 1, D, D, seed=15, pos=[L - n - 3])
    q_ref, k_ref, v_ref = swa.swa_qk_norm_rope(**c)
    kc = torch.zeros((1, 1, L, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    q = swa.swa_qk_norm_rope_append(**c, k_cache=kc, v_cache=vc,
                                    seq_lens=torch.tensor([L], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    p = L - n - 3
    assert torch.equal(q, q_ref)
    for cache, rows in ((kc, k_ref), (vc, v_ref)):
        assert torch.equal(cache[0, 0, p:p + n], rows[0, :, 0])
        assert not cache[0, 0, p + n:].any() and not cache[0, 0, p - 1000:p].any()
    # one token every 2^30 elements
    flat = vc.view(-1)
    step = 1 << 30
    strided = flat.as_strided((1, 2, 2, D), (2 * step, step, D, 1), 512)
    strided.copy_(c["q"][:, :2])
    got = swa.swa_qk_norm_rope(strided, c["k"][:, :2], c["v"][:, :2], c["q_weight"], c["k_weight"],
                               1e-6, c["inv_freq"], c["q_pos"])[0]
    torch.cuda.synchronize()
    assert torch.equal(got, q_ref[:, :2])
