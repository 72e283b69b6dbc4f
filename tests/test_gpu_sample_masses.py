"""sample_logits where |logit| / T is large, and where a row is all ties: what a mass is off by shows in the log probability alone."""
import math

import pytest
import torch

import speculative_decoding_verification_spec_gb300 as sv

from test_gpu_sample import DT, F32, check, settings, uniforms

pytestmark = pytest.mark.gpu

# a few rows (clusters) and many (a CTA each)
ROWS = [4, 160]
WAYS = {"free": {}, "k5": dict(k=5), "k700": dict(k=700), "p": dict(p=0.9), "k700_p": dict(k=700, p=0.9), "minp": dict(mp=0.01)}


def far(g, N, V, dtype):
    """Rows whose largest logit lies anywhere from 20 to 1000 from zero, on either side, over temperatures from 1e-3 to 0.3."""
    top = 20.0 * 50.0 ** torch.rand(N, generator=g) * torch.where(torch.arange(N) % 2 == 0, 1.0, -1.0)
    T = 1e-3 * 300.0 ** torch.rand(N, generator=g)
    # cases with |top| / T log2(e) near 10^4
    top[:4], T[:4] = torch.tensor([30.0, 90.0, 124.0, 968.0])[:N], torch.tensor([0.005, 0.01, 0.01117, 0.09])[:N]
    top = top.to(DT[dtype]).float()
    return top, T


@pytest.mark.parametrize("N", ROWS)
@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_token_is_certain(dtype, way, N):
    """The others have no mass: the log probability is 0.  With a mass right to 2^-28 what is left are the roundings of a sum next to zero and
    of a logarithm's argument and value, 2^-25 each, and the logarithm's own 2^-24: under 2^-22."""
    g = torch.Generator().manual_seed(40)
    V = 9001
    for _ in range(3):
        top, T = far(g, N, V, dtype)
        x = (top[:, None] - 200 * T[:, None] - 0.1 * top[:, None].abs() - 30 * torch.rand(N, V, generator=g)).to(DT[dtype])
        at = torch.randint(0, V, (N,), generator=g)
        x[torch.arange(N), at] = top.to(DT[dtype])
        r = sv.sample_logits(x.cuda(), uniforms(g, N).cuda(), **settings(N, T, **WAYS[way]))
        assert r["tokens"].tolist() == at.tolist()
        assert float(r["logprob"].abs().max()) <= 2.0 ** -22


@pytest.mark.parametrize("N", ROWS)
@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_that_lie_near(dtype, way, N):
    """Some twenty tokens share the mass, ties among them, and many lie some steps of the type below."""
    g = torch.Generator().manual_seed(41)
    V = 9001
    top, T = far(g, N, V, dtype)
    x = top[:, None] - T[:, None] * (15 + 60 * torch.rand(N, V, generator=g))
    near = torch.randperm(V, generator=g)[:20]
    x[:, near] = top[:, None] - T[:, None] * 4 * torch.rand(N, 20, generator=g)
    x[:, near[:3]] = top[:, None]
    check(x.to(DT[dtype]).cuda(), uniforms(g, N), T=T, exempt=1, **WAYS[way])


@pytest.mark.parametrize("N", [3, 130])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value,T", [(0.0, 1.0), (90.0, 0.01), (1.0, 2.880), (-124.0, 0.01117)])
def test_a_whole_row_of_ties(value, T, dtype, N):
    """The widest row there is, all of one value: a thread's partial sums are the largest that they can be.  Every token has the same mass."""
    V = 262144
    x = torch.full((1, V), value, dtype=DT[dtype], device="cuda").expand(N, -1).contiguous()
    j = (torch.arange(N) * (V // N) + 1).clamp(max=V - 1)
    u = ((j.double() + 0.5) / V).float()
    for kw in ({}, dict(p=0.5), dict(k=9), dict(mp=0.5), dict(k=1000, p=0.9)):
        r = sv.sample_logits(x, u.to(F32).cuda(), **settings(N, T, **kw))
        assert r["tokens"].tolist() == j.tolist()
        assert float((r["logprob"].cpu() + math.log(V)).abs().max()) <= 2.0 ** -22 * (1 + math.log(V))
