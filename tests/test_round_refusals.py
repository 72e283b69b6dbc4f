"""The calls around the verify step refuse bad arguments on the host, and the 64-bit references they are tested against
hold what they should."""
import ctypes
import math

import pytest
import torch

import speculative_decoding_verification_spec_gb300 as sv
from speculative_decoding_verification_spec_gb300 import build_ext

import round_ref as R


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return sv.load()


P = ctypes.c_void_p
F = ctypes.c_float
fake, odd = P(0x10000), P(0x10002)   # never dereferenced: validation fails first
INVALID, WORKSPACE = 1, 3


def test_process_logits_refusals(lib):
    def call(x=fake, y=fake, dt=1, B=2, Rr=3, V=100, N=2, tok=fake, par=None, H=0, hist=None, pl=None, nb=0, bt=None, bv=None,
             al=None, ins=None, outs=None):
        return lib.process_logits(x, y, dt, B, Rr, V, ins, outs, tok, par, N, hist, H, pl, None, None, None, None, bt, bv, nb, al,
                                  None, None)

    assert call(B=0) == 0
    st = lambda *a: (ctypes.c_int64 * 2)(*a)
    for bad in (dict(B=-1), dict(B=65536), dict(Rr=0), dict(Rr=4), dict(V=0), dict(N=-1), dict(N=4097), dict(dt=2), dict(dt=7),
                dict(x=None), dict(y=None), dict(tok=None), dict(tok=odd), dict(par=odd), dict(H=5), dict(H=-1), dict(pl=odd),
                dict(nb=3), dict(nb=3, bt=fake), dict(nb=-1), dict(al=odd), dict(ins=st(-1, 100)), dict(outs=st(300, 50)),
                dict(outs=st(250, 100)), dict(ins=st(600, 200))):
        assert call(**bad) == INVALID, bad


def test_cache_refusals(lib):
    def write(k=fake, v=fake, dt=1, B=2, T=4, H=2, D=64, kc=fake, vc=fake, ks=fake, vs=fake, pages=8, page=16, tab=fake, width=4,
              lens=fake, acc=None, nodes=None, nw=0, lo=None):
        return lib.kv_cache_write(k, None, v, None, dt, B, T, H, D, kc, vc, ks, vs, pages, page, tab, width, lens, acc, nodes, nw,
                                  lo, None, None)

    assert write(B=0) == 0
    for bad in (dict(B=-1), dict(T=0), dict(H=0), dict(D=96), dict(D=256), dict(page=8), dict(page=48), dict(page=256), dict(pages=0),
                dict(width=0), dict(dt=5), dict(k=None), dict(v=None), dict(kc=P(0x10008)), dict(vc=None), dict(ks=None),
                dict(vs=odd), dict(tab=None), dict(lens=None), dict(acc=odd), dict(nodes=fake, nw=3), dict(lo=fake),
                dict(width=1 << 28), dict(k=P(0x10001))):
        assert write(**bad) == INVALID, bad

    def read(B=2, n=5, dt=1, ko=fake, vo=fake, start=None, D=64, page=16):
        return lib.kv_cache_read(fake, fake, fake, fake, 8, page, 2, D, fake, 4, fake, start, B, n, ko, vo, dt, None, None)

    assert read(B=0) == 0
    for bad in (dict(B=-1), dict(n=0), dict(dt=4), dict(ko=None), dict(vo=P(0x10008)), dict(start=odd), dict(D=80), dict(page=0)):
        assert read(**bad) == INVALID, bad


def test_attention_refusals(lib):
    need = lib.verify_attention_workspace_bytes(2, 4, 8, 2, 64)
    assert need > 0 and need % 16 == 0
    for sizes in ((-1, 4, 8, 2, 64), (2, 0, 8, 2, 64), (2, 257, 8, 2, 64), (2, 4, 9, 2, 64), (2, 4, 8, 0, 64), (2, 4, 8, 2, 96)):
        assert lib.verify_attention_workspace_bytes(*sizes) == 0, sizes

    def call(q=fake, k=fake, v=fake, dt=1, B=2, T=4, hq=8, hkv=2, D=64, s=0.125, out=fake, lse=None, par=None, ws=fake, wsb=need,
             lens=fake, nr=None):
        return lib.verify_attention(q, None, k, None, v, None, dt, B, T, hq, hkv, D, fake, fake, fake, fake, 8, 16, fake, 4, lens,
                                    par, nr, F(s), out, lse, None, ws, wsb, None)

    assert call(B=0) == 0
    for bad in (dict(B=-1), dict(T=0), dict(T=257), dict(hq=9), dict(hq=1), dict(hkv=0), dict(D=72), dict(dt=0), dict(dt=9),
                dict(s=0.0), dict(s=math.inf), dict(s=math.nan), dict(q=None), dict(k=None), dict(v=None), dict(out=None),
                dict(out=P(0x10008)), dict(lse=odd), dict(par=odd), dict(lens=None), dict(nr=odd)):
        assert call(**bad) == INVALID, bad
    assert call(ws=None) == WORKSPACE
    assert call(ws=P(0x10008)) == WORKSPACE
    assert call(wsb=need - 1) == WORKSPACE


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    c = sv.kv_cache(2, 1, 16, 64, device="cpu")
    assert c.k.shape == (2, 1, 16, 64) and c.k_scale.shape == (2, 1)
    i32 = dict(dtype=torch.int32)
    q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    tab, lens = torch.zeros(1, 1, **i32), torch.zeros(1, **i32)
    for f in (lambda: sv.verify_attention(q, c, tab, lens), lambda: sv.kv_cache_read(c, tab, lens, max_len=3),
              lambda: sv.kv_cache_write(q[:, :, :1], q[:, :, :1], c, tab, lens),
              lambda: sv.process_logits(torch.zeros(1, 1, 8))):
        with pytest.raises(sv.SpecVerifyError):
            f()


def test_reference_codes_are_e4m3():
    """The reference's grid is torch's e4m3 type: every code is a fixed point, and values round alike."""
    codes = torch.arange(256, dtype=torch.uint8).view(R.FP8).float()
    ok = ~codes.isnan()
    assert bool((R.quantise(codes[ok], 0) == codes[ok].double()).all())
    x = torch.randn(20000, generator=torch.Generator().manual_seed(1)) * torch.logspace(-4, 2.2, 20000)
    assert bool((R.quantise(x, 0) == x.to(R.FP8).double())[x.abs() <= 448].all())
    assert bool(R.quantise(x, 0)[x.abs() > 448].isnan().all())
    assert R.scale_exp(448.0) == 0 and R.scale_exp(448.1) == 1 and R.scale_exp(0.0) == -60 and R.scale_exp(1e38) == 60


def test_reference_attention_is_softmax():
    g = torch.Generator().manual_seed(2)
    q, k, v = torch.randn(2, 4, 64, generator=g), torch.randn(9, 2, 64, generator=g).double(), torch.randn(9, 2, 64, generator=g).double()
    out, lse, *_ = R.attention_ref(q, k, v, None, None, None, 2, 0.125)
    s = torch.einsum("thd,jhd->thj", q.double(), k.repeat_interleave(2, 1)) * 0.125
    want = torch.einsum("thj,jhd->thd", torch.softmax(s, -1), v.repeat_interleave(2, 1))
    assert torch.allclose(out, want, rtol=1e-12, atol=1e-12) and torch.allclose(lse, torch.logsumexp(s, -1))
    assert R.path(None, 3) == [3, 2, 1, 0] and R.path(torch.tensor([-1, -1, 0, 2]), 4) == [4, 3, 1, 0]
