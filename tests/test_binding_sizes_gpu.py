"""The binding refuses tensors that a call would run past, on the paged and
the fused-append attention; larger ones serve."""
import pytest
import torch

pytestmark = pytest.mark.gpu

B, Q, HQ, HKV, D, L = 3, 4, 4, 2, 128, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


def _tensors():
    g = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    pos = torch.tensor([0, 5, 60], dtype=torch.int32).cuda()
    return dict(q=rnd(B, Q, HQ, D), k_new=rnd(B, Q, HKV, D), v_new=rnd(B, Q, HKV, D),
                k=rnd(B, HKV, L, D), v=rnd(B, HKV, L, D), seq_lens=pos + Q, q_pos=pos,
                out=torch.empty((B, Q, HQ, D), dtype=torch.bfloat16, device="cuda"),
                lse=torch.empty((B, Q, HQ), device="cuda"))


def _call(entry, t):
    import sliding_window_speculative_gb300 as swa
    s = D ** -0.5
    if entry == "append":
        return swa.swa_append_verify_attn(t["q"], t["k_new"], t["v_new"], t["k"], t["v"],
                                          t["seq_lens"], t["q_pos"], 20, s, out=t["out"], lse=t["lse"])
    table = torch.arange(B * L // 16, dtype=torch.int32).view(B, L // 16).cuda()
    k, v = (t[n].view(B, HKV, L // 16, 16, D).transpose(1, 2).reshape(-1, HKV, 16, D).contiguous()
            for n in ("k", "v"))
    return swa.swa_verify_attn_paged(t["q"], k, v, table, t["seq_lens"], t["q_pos"], 20, s,
                                     out=t["out"], lse=t["lse"])


@pytest.mark.parametrize("entry", ["paged", "append"])
@pytest.mark.parametrize("name", ["seq_lens", "q_pos", "out", "lse"])
def test_short_tensors_are_refused_and_long_ones_serve(entry, name):
    t = _tensors()
    short = dict(t, **{name: t[name][:B - 1].contiguous()})
    with pytest.raises(ValueError, match=f"{name} needs"):
        _call(entry, short)
    want = [x.clone() for x in _call(entry, t)]
    got = _call(entry, dict(t, **{name: torch.cat([t[name], t[name][:1]])}))
    torch.cuda.synchronize()
    assert all(torch.equal(g[:B], w) for g, w in zip(got, want))


def test_an_append_needs_a_slab_per_sequence():
    t = _tensors()
    with pytest.raises(ValueError, match="one slab per sequence"):
        _call("append", dict(t, k=t["k"][:2].contiguous(), v=t["v"][:2].contiguous()))
