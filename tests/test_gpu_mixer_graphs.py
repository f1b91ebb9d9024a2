"""Packed calls of linear attention and window attention in one captured graph, replayed with other offsets than those of
the capture: sequences are cut, split and masked by what the offsets say then, and every replay is the eager call."""
import os

import pytest
import torch

from selective_state_space_47_amd import _build, binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TOKENS = 1400
# sequences of many lengths, empty ones, a gap before and behind
OFFSETS = [[0, 1300, 1300, 1400], [0, 100, 101, 1400], [7, 8, 650, 1290], [0, 0, 0, 0], [3, 67, 131, 195]]


@pytest.fixture(scope="module", autouse=True)
def _native():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(_build.LIB_PATH):
        _build.build()
    binding.lib()


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_other_offsets_at_replay(io):
    print(f"[mixer graphs] {io}", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(io)  # noqa: E731
    hk, hv, d = 2, 40, 16
    x = dict(q=n(TOKENS, hk, d), k=n(TOKENS, hk, d), v=n(TOKENS, hv, d), do=n(TOKENS, hv, d),
             g=-torch.rand(TOKENS, hv, generator=gen, device=DEV), s=torch.randn(3, hv, d, d, generator=gen, device=DEV),
             wq=n(TOKENS, 6, 64), wk=n(TOKENS, 2, 64), wv=n(TOKENS, 2, 64), wdo=n(TOKENS, 6, 64))
    offsets = torch.tensor(OFFSETS[0], device=DEV)

    def call():
        out, last = binding.mamba_linear_attn_fwd(x["q"], x["k"], x["v"], x["g"], initial_state=x["s"],
                                                  seq_offsets=offsets, return_last_state=True)
        a = binding.mamba_linear_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], initial_state=x["s"],
                                          seq_offsets=offsets, dlast=x["s"])
        w, lse = binding.mamba_window_attn_fwd(x["wq"], x["wk"], x["wv"], 100, 3, seq_offsets=offsets, return_lse=True)
        b = binding.mamba_window_attn_bwd(x["wq"], x["wk"], x["wv"], w, lse, x["wdo"], 100, 3, seq_offsets=offsets)
        caches = [torch.zeros(3, 103, 2, 64, device=DEV, dtype=io) for _ in range(2)]
        binding.mamba_window_cache_store(*caches, x["wk"], x["wv"], 3, seq_offsets=offsets)
        tokens = dict(out=out, w=w, lse=lse, **{"l" + m: a[m] for m in ("dq", "dk", "dv", "dg")},
                      **{"w" + m: b[m] for m in ("dq", "dk", "dv")})
        return tokens, dict(last=last, ds=a["dinitial_state"], kc=caches[0], vc=caches[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens, whole = call()
    for off in OFFSETS + OFFSETS[::-1]:
        offsets.copy_(torch.tensor(off, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        want_tokens, want_whole = call()
        for name, t in tokens.items():
            assert torch.equal(t[off[0]:off[-1]], want_tokens[name][off[0]:off[-1]]), (off, name)
        for name, t in whole.items():
            assert torch.equal(t, want_whole[name]), (off, name)
        if off[0] == off[-1]:
            assert torch.equal(whole["last"], x["s"]) and torch.equal(whole["ds"], x["s"])
            assert not bool(whole["kc"].any())
