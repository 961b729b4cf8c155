"""The layer's calls with an explicit stream inside a capture, and on a side
stream whose results another stream uses (CUDA path through the C ABI)."""
import numpy as np
import pytest
import torch

import workloads
from tests.gpu_helpers import bits, lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def agb():
    return lib()


@pytest.mark.parametrize("raw", [False, True])
def test_an_explicit_stream_in_a_capture(agb, raw):
    rng = np.random.default_rng(1)
    N, H = 300, 64
    src, dst = (torch.as_tensor(rng.integers(0, N, 4000).astype(np.int32)).to(DEV) for _ in range(2))
    g = agb.ag_graph_lower(src, dst, N)
    A, B, V, G = (workloads.features(N, H, torch.bfloat16, k, DEV) for k in range(4))
    lam, one = torch.full((2,), 0.4, device=DEV), torch.ones(H, device=DEV)
    pos, freq = torch.arange(N, device=DEV), agb.ag_rotary_freqs(16)[0].to(DEV)

    def step(stream):
        kw = dict(p=0.1, seed=3, stream=stream)
        q, k = agb.ag_rotary(A, B, pos, freq, 4, stream=stream)
        y, lse = agb.ag_diff_attn_fwd(g, q, k, V, lam, 0.25, **kw)
        x, z = agb.ag_resnorm_fwd(A, y, G, gamma1=one, gamma2=one, **kw)
        d = agb.ag_resnorm_backward(x, y, G, z, x, gamma1=one, gamma2=one, **kw)
        return [q, k, y, lse, x, z, agb.ag_dropout(z, **kw)] + [d[n] for n in sorted(d)] + list(
            agb.ag_diff_attn_backward(g, q, k, V, lam, 0.25, lse, d["B"], **kw))
    want = step(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    name = s.cuda_stream if raw else s
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg, stream=s):
        out = step(name)
    for t in out:
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(2):
        cg.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(out, want))
    # eager on the side stream; its results are used on this one after a wait, and its scratch is given back in between
    for _ in range(20):
        got = step(name)
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))
