"""sample_logits where a grammar leaves fewer tokens than top-k asks for, the others masked by a large finite number or by -inf."""
import math

import pytest
import torch

from test_gpu_sample import DT, check, logits, uniforms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [4, 160])
@pytest.mark.parametrize("mask", ["-1e9", "lowest", "-inf"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_fewer_tokens_than_top_k(dtype, mask, N):
    g = torch.Generator().manual_seed(50)
    V = 12007
    low = {"-1e9": -1e9, "lowest": torch.finfo(DT[dtype]).min, "-inf": -math.inf}[mask]
    x = logits(g, N, V, dtype)
    legal = torch.zeros(N, V, dtype=torch.bool)
    for r in range(N):
        legal[r, torch.randperm(V, generator=g)[:1 + 3 * r % 40]] = True
    x = torch.where(legal, x, torch.tensor(low, dtype=DT[dtype]))
    for kw in (dict(k=50), dict(k=700), dict(k=50, p=0.9), dict(k=700, p=0.9, T=0.5), dict(p=0.9), dict(k=50, mp=0.01), dict(mp=1e-4)):
        out = check(x.cuda(), uniforms(g, N), exempt=1, **kw)
        assert bool(legal.gather(1, out["tokens"].cpu().long()[:, None]).all())
