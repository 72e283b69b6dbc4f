"""The calls around the verify step look at where every tensor lives before anything is launched.  CPU tensors that claim a
device stand in for CUDA ones; nothing here reaches a kernel."""
import pytest
import torch

import speculative_decoding_verification_spec_gb300 as sv
from speculative_decoding_verification_spec_gb300 import binding, build_ext


class On(torch.Tensor):
    """A CPU tensor that says it is on cuda:0."""
    at = 0

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.at


class OnNext(On):
    at = 1


def on(t):
    return None if t is None else t.as_subclass(On)


class Reached(Exception):
    pass


class Lib:
    def verify_attention_workspace_bytes(self, *a):
        return 256

    def __getattr__(self, name):
        def call(*a):
            raise Reached(name)
        return call


@pytest.fixture(autouse=True)
def host(monkeypatch):
    """No launch: the library raises once a call has passed its checks."""
    monkeypatch.setattr(binding, "load", lambda *a: Lib())
    monkeypatch.setattr(binding, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(binding, "_raw_stream", lambda stream, at: 0)


I32, F32, BF = torch.int32, torch.float32, torch.bfloat16
z = lambda *s, dtype=F32: on(torch.zeros(s, dtype=dtype))


class Ws:
    def __init__(self, t):
        self.t = t

    def get(self, n):
        return self.t


def cases():
    """name -> (function, tensors by argument)."""
    cache = dict(ck=z(4, 2, 16, 64, dtype=torch.uint8), cv=z(4, 2, 16, 64, dtype=torch.uint8), ks=z(4, 2), vs=z(4, 2),
                 table=z(3, 2, dtype=I32), lens=z(3, dtype=I32))
    c = lambda a: (a["ck"], a["cv"], a["ks"], a["vs"])

    def attention(a):
        return sv.verify_attention(a["q"], c(a), a["table"], a["lens"], k=a["k"], v=a["v"], parents=a["parents"], n_rows=a["n_rows"],
                                   out=dict(out=a["out"], lse=a["lse"], row_status=a["row_status"]), workspace=Ws(a["workspace"]))

    def write(a):
        return sv.kv_cache_write(a["k"], a["v"], c(a), a["table"], a["lens"], accepted_len=a["accepted"], out_nodes=a["nodes"],
                                 out=dict(lens=a["lens_out"], row_status=a["row_status"]))

    def read(a):
        return sv.kv_cache_read(c(a), a["table"], a["lens"], max_len=7, start=a["start"],
                                out=dict(k=a["k"], v=a["v"], row_status=a["row_status"]))

    def logits(a):
        kw = {n: a[n] for n in a if n not in ("logits", "out", "row_status")}
        return sv.process_logits(a["logits"], out=dict(logits=a["out"], row_status=a["row_status"]), **kw)

    yield attention, dict(cache, q=z(3, 5, 4, 64, dtype=BF), k=z(3, 5, 2, 64, dtype=BF), v=z(3, 5, 2, 64, dtype=BF), parents=z(3, 4, dtype=I32),
                          n_rows=z(3, dtype=I32), out=z(3, 5, 4, 64, dtype=BF), lse=z(3, 5, 4), row_status=z(3, dtype=I32),
                          workspace=z(256, dtype=torch.uint8))
    yield write, dict(cache, k=z(3, 5, 2, 64, dtype=BF), v=z(3, 5, 2, 64, dtype=BF), accepted=z(3, dtype=I32), nodes=z(3, 4, dtype=I32),
                      lens_out=z(3, dtype=I32), row_status=z(3, dtype=I32))
    yield read, dict(cache, start=z(3, dtype=I32), k=z(3, 7, 2, 64, dtype=BF), v=z(3, 7, 2, 64, dtype=BF), row_status=z(3, dtype=I32))
    yield logits, dict(logits=z(3, 4, 50), out=z(3, 4, 50), row_status=z(3, dtype=I32), tokens=z(3, 3, dtype=I32), parents=z(3, 3, dtype=I32),
                       history=z(3, 9, dtype=I32), prompt_len=z(3, dtype=I32), history_len=z(3, dtype=I32), repetition=z(3), presence=z(3),
                       frequency=z(3), bias_tokens=z(3, 2, dtype=I32), bias_values=z(3, 2), allowed=z(3, 4, 2, dtype=I32))


@pytest.mark.parametrize("i", range(4))
def test_every_tensor_has_to_be_on_the_call_s_device(i):
    f, args = list(cases())[i]
    with pytest.raises(Reached):
        f(args)
    for name, t in args.items():
        with pytest.raises(sv.SpecVerifyError):
            f(dict(args, **{name: t.as_subclass(torch.Tensor)}))
        with pytest.raises(ValueError):
            f(dict(args, **{name: t.as_subclass(OnNext)}))


@pytest.mark.parametrize("i", range(4))
def test_the_device_has_to_be_the_current_one(i, monkeypatch):
    f, args = list(cases())[i]
    monkeypatch.setattr(binding, "_current_device", lambda: 1)
    with pytest.raises(ValueError):
        f(args)


@pytest.mark.parametrize("i", range(3))
def test_codes_have_to_be_e4m3(i):
    f, args = list(cases())[i]
    for name in ("ck", "cv"):
        for dtype in (torch.int8, torch.bool, torch.float8_e5m2, torch.int16):
            with pytest.raises(TypeError):
                f(dict(args, **{name: args[name].to(dtype)}))
        with pytest.raises(Reached):
            f(dict(args, **{name: args[name].view(torch.float8_e4m3fn)}))


def test_the_workspace_is_that_of_the_rows(monkeypatch):
    monkeypatch.undo()
    build_ext.build()
    need = lambda T, hq, hkv, D: sv.load().verify_attention_workspace_bytes(1, T, hq, hkv, D)
    for D in (64, 128):
        assert need(1, 32, 8, D) <= 9 << 20 and need(256, 64, 1, D) <= 22 << 20
        for hq, hkv in ((1, 1), (8, 2), (40, 8), (64, 4)):
            sizes = [need(T, hq, hkv, D) for T in range(1, 257)]
            assert sizes == sorted(sizes) and all(n % 16 == 0 for n in sizes)


def test_the_stream_has_to_be_on_the_call_s_device(monkeypatch):
    monkeypatch.undo()

    class Stream:
        device_index, cuda_stream = 1, 5

    assert binding._raw_stream(Stream(), 1) == 5
    with pytest.raises(ValueError):
        binding._raw_stream(Stream(), 0)
