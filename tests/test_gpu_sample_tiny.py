"""sample_logits on bf16 rows whose largest logit is positive and so small that the first sweep's counts have no place for it, at temperatures
small enough to tell it from zero."""
import math

import pytest
import torch

from test_gpu_sample import check, uniforms

pytestmark = pytest.mark.gpu

WAYS = {"p": dict(p=0.9), "p_high": dict(p=0.9999), "k700": dict(k=700), "k700_p": dict(k=700, p=0.8), "p_minp": dict(p=0.9, mp=0.01)}


# few rows (clusters) and many (a CTA each)
@pytest.mark.parametrize("N", [4, 160])
@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("rest", ["masked", "zeros", "below", "smaller", "ties"])
def test_largest_logits_under_every_place(rest, way, N):
    g = torch.Generator().manual_seed(60)
    V = 3001
    for heat in (1e-8, 1e-3, 0.02, 0.05, 0.3, 2.0):  # of the largest logit: from certain tokens to rows where all weigh alike
        top = 10.0 ** (-7 - 20 * torch.rand(N, generator=g))  # 64 / 2^31 is 3e-8: some lie over it
        x = torch.randn(N, V, generator=g)
        if rest == "masked":
            x = torch.full((N, V), -math.inf)
        elif rest == "zeros":
            x = torch.where(x > 0, 0.0, -0.0)
        elif rest == "below":
            x = -x.abs()
        else:
            x = top[:, None] * torch.rand(N, V, generator=g)
        x = torch.minimum(x, 0.99 * top[:, None])
        at = torch.randint(0, V, (N,), generator=g)
        x[torch.arange(N), at] = top
        if rest == "ties":
            x[:, ::7] = top[:, None]
        x = x.bfloat16()
        T = (heat * x.float().amax(1)).clamp(min=1e-30)
        check(x.cuda(), uniforms(g, N), T=T, exempt=2, **WAYS[way])
