"""The calls around the verify step against plain 64-bit references: the 8-bit cache (write, read), attention over it,
and logit processing."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_spec_gb300 as sv
from speculative_decoding_verification_spec_gb300 import binding as B_

import round_ref as R
from parity import Guarded

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def same(a, b):
    """Equal values, NaN where NaN."""
    a, b = a.double(), b.double()
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


class Pool:
    """A cache on the GPU whose requests hold `lens` tokens, in scattered pages; the rest of the pool, and the slots
    past the lengths, hold NaN codes and the spare pages' scales NaN, none of which may be interpreted."""

    def __init__(self, g, lens, hkv, page, D, spare=0, spread=1.0):
        per = [-(-(n + spare) // page) for n in lens]
        P = sum(per) + 3
        self.lens, self.page = lens, page
        perm = torch.randperm(P, generator=g)
        width = max(1, max(per))
        self.table = torch.full((len(lens), width), -7, dtype=torch.int32)  # unused entries are no page
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = perm[at:at + n].to(torch.int32)
            at += n
        self.codes, self.scales = [], []
        for _ in range(2):
            c = torch.full((P, hkv, page, D), math.nan).to(R.FP8)
            s = torch.full((P, hkv), math.nan)
            for b, n in enumerate(lens):
                for i in range(0, n, page):
                    p = int(self.table[b, i // page])
                    m = min(page, n - i)
                    raw = torch.randn(hkv, m, D, generator=g) * 60
                    c[p, :, :m] = raw.clamp(-448, 448).to(R.FP8)
                    s[p] = torch.exp2(torch.randint(-9, -4, (hkv,), generator=g).float() * spread)
            self.codes.append(c)
            self.scales.append(s)
        dev = lambda x: x.view(torch.uint8).cuda().view(R.FP8)
        self.cache = sv.KVCache(dev(self.codes[0]), dev(self.codes[1]), self.scales[0].cuda(), self.scales[1].cuda())
        self.dtable, self.dlens = self.table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")

    def line(self, which, b):
        return R.line(self.codes[which].float(), self.scales[which], self.table[b], self.lens[b])


# ------------------------------------------------------------------ read

@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("page,D,hkv", [(16, 64, 1), (32, 128, 3), (64, 128, 8), (128, 64, 2)])
def test_read_back(dtype, page, D, hkv):
    g = torch.Generator().manual_seed(page + D)
    p = Pool(g, [0, 1, page, page + 1, 3 * page - 5], hkv, page, D)
    n = 3 * page - 3
    gd = Guarded()
    out = dict(k=gd.empty((5, n, hkv, D), DT[dtype], "k"), v=gd.empty((5, n, hkv, D), DT[dtype], "v"),
               row_status=gd.empty((5,), torch.int32, "status"))
    sv.kv_cache_read(p.cache, p.dtable, p.dlens, max_len=n, dtype=DT[dtype], out=out)
    torch.cuda.synchronize()
    gd.check()
    assert out["row_status"].tolist() == [0] * 5
    for which, name in enumerate("kv"):
        for b, length in enumerate(p.lens):
            want = torch.zeros(n, hkv, D, dtype=torch.float64)
            m = min(n, length)
            want[:m] = p.line(which, b)[:m]
            assert same(out[name][b].cpu(), want.to(DT[dtype]))


def test_read_window_and_bad_pages():
    g = torch.Generator().manual_seed(5)
    p = Pool(g, [100, 40, 70, 16, 16], 2, 16, 64)
    start = torch.tensor([90, 0, 33, 0, -1], dtype=torch.int32, device="cuda")
    p.dtable[2, 2] = 10 ** 6       # tokens 32 .. 47
    p.dlens[3] = 10 ** 6           # more than the table's row holds
    r = sv.kv_cache_read(p.cache, p.dtable, p.dlens, max_len=20, start=start, dtype=torch.float32)
    assert r["row_status"].tolist() == [0, 0, B_.ROW_BAD_PAGE, B_.ROW_BAD_LENGTH, B_.ROW_BAD_LENGTH]
    k = r["k"].cpu().double()
    a = p.line(0, 0)
    assert same(k[0, :10], a[90:]) and bool((k[0, 10:] == 0).all())
    assert same(k[1], p.line(0, 1)[:20])
    assert bool(k[2, :15].isnan().all()) and same(k[2, 15:], p.line(0, 2)[48:53])
    assert bool(k[3].isnan().all()) and bool(k[4].isnan().all())


# ------------------------------------------------------------------ write

def check_write(p, k, v, accepted=None, nodes=None, bad=()):
    T = k.shape[1]
    gd = Guarded()
    B = len(p.lens)
    cc = [gd.empty(p.codes[0].shape, torch.uint8, "codes%d" % i) for i in range(2)]
    ss = [gd.empty(p.scales[0].shape, torch.float32, "scale%d" % i) for i in range(2)]
    for i in range(2):
        cc[i].copy_(p.codes[i].view(torch.uint8))
        ss[i].copy_(p.scales[i])
    out = dict(lens=gd.empty((B,), torch.int32, "lens"), row_status=gd.empty((B,), torch.int32, "status"))
    cache = sv.KVCache(cc[0].view(R.FP8), cc[1].view(R.FP8), ss[0], ss[1])
    acc = None if accepted is None else torch.tensor(accepted, dtype=torch.int32, device="cuda")
    nd = None if nodes is None else nodes.cuda()
    for _ in range(2):  # a second call on the same lengths finds the codes and scales as it would write them
        r = sv.kv_cache_write(k, v, cache, p.dtable, p.dlens, accepted_len=acc, out_nodes=nd, out=out)
        torch.cuda.synchronize()
        gd.check()
        lens = list(p.lens)
        for which, x in enumerate((k.cpu(), v.cpu())):
            codes, scales = p.codes[which].double(), p.scales[which].double()
            for b in range(B):
                if b in bad:
                    continue
                rows = R.accepted_rows(T, None if accepted is None else accepted[b], None if nodes is None else nodes[b])
                R.write_ref(codes, scales, x[b], p.table[b], p.lens[b], rows)
                lens[b] = p.lens[b] + len(rows)
            assert same(cache[2 + which].cpu(), scales)
            assert same(cache[which].cpu().view(torch.uint8).view(R.FP8).float(), codes)
        assert r["lens"].tolist() == lens
    return r


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("page,D,hkv,T", [(16, 64, 1, 1), (16, 128, 2, 5), (32, 64, 3, 33), (64, 128, 2, 7), (128, 128, 1, 200),
                                          (128, 64, 2, 129)])
def test_write(dtype, page, D, hkv, T):
    g = torch.Generator().manual_seed(page * D + T)
    p = Pool(g, [0, 1, page - 1, page, 2 * page - 3], hkv, page, D, spare=T)
    mag = torch.exp2(torch.randint(-6, 7, (5, T, 1, 1), generator=g).float())
    k, v = ((torch.randn(5, T, hkv, D, generator=g) * mag).to(DT[dtype]).cuda() for _ in range(2))
    r = check_write(p, k, v)
    assert r["row_status"].tolist() == [0] * 5


@pytest.mark.parametrize("tree", [False, True])
def test_write_accepted_rows(tree):
    g = torch.Generator().manual_seed(11)
    T, hkv, D, page = 9, 2, 128, 16
    lens = [0, 15, 16, 30, 7, 12]
    acc = [-1, 0, 3, 8, 5, 2]
    p = Pool(g, lens, hkv, page, D, spare=T)
    k, v = (torch.randn(6, T, hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
    nodes = None
    if tree:
        nodes = torch.full((6, T - 1), -1, dtype=torch.int32)
        for b, a in enumerate(acc):
            if a > 0:
                nodes[b, :a] = torch.randperm(T - 1, generator=g)[:a].sort().values.to(torch.int32)
    check_write(p, k, v, acc, nodes)


def test_write_strided_and_unaligned_rows():
    g = torch.Generator().manual_seed(12)
    p = Pool(g, [3, 20], 2, 16, 64, spare=5)
    big = torch.randn(2, 2, 5, 3 * 64 + 1, generator=g).bfloat16().cuda()   # [B, H, T, ...]
    k = big[..., 1:65].transpose(1, 2)
    v = big[..., 64:128].transpose(1, 2)
    assert not k.is_contiguous()
    check_write(p, k, v)


def test_write_special_values():
    g = torch.Generator().manual_seed(13)
    p = Pool(g, [0, 4], 1, 16, 64, spare=6)
    k = torch.randn(2, 6, 1, 64, generator=g)
    k[0, 0, 0, 0] = math.nan
    k[0, 1, 0, 1] = math.inf
    k[0, 2, 0, 2] = -math.inf
    k[0, 3] = 0.0
    k[1, 0, 0, :4] = torch.tensor([1e30, -1e30, 448.0 * 2.0 ** 60, 3.0])
    v = torch.zeros(2, 6, 1, 64)                       # a block of zeros takes the smallest scale
    v[1, 2, 0, 5] = 2.0 ** -80
    check_write(p, k.cuda(), v.cuda())


def test_write_scale_is_the_smallest_that_holds():
    """Magnitudes on and next to 448 * 2^e."""
    lens, T = [0] * 4, 1
    for e in (-60, -20, 0, 7):
        p = Pool(torch.Generator().manual_seed(e + 100), lens, 1, 16, 64, spare=T)
        k = torch.zeros(4, T, 1, 64)
        for b, a in enumerate((448.0, np.nextafter(np.float32(448), np.float32(0)), np.nextafter(np.float32(448), np.float32(500)), 449.0)):
            k[b, 0, 0, b] = float(a) * 2.0 ** e
        check_write(p, k.cuda(), (-k).cuda())


def test_write_refuses_bad_requests_whole():
    g = torch.Generator().manual_seed(14)
    T = 20
    p = Pool(g, [3, 5, 8, 16, 2], 2, 16, 64, spare=T)
    k, v = (torch.randn(5, T, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    p.table[1, 1] = p.codes[0].shape[0]           # the second page of request 1
    p.dtable = p.table.cuda()
    p.dlens = torch.tensor([3, 5, -1, 16, 2], dtype=torch.int32, device="cuda")
    p.lens = [3, 5, -1, 16, 2]
    acc = [19, 19, 4, 25, 3]
    r = check_write(p, k, v, acc, bad=(1, 2, 3))
    assert r["row_status"].tolist() == [0, B_.ROW_BAD_PAGE, B_.ROW_BAD_LENGTH, B_.ROW_BAD_LENGTH, 0]
    nodes = torch.full((5, T - 1), -1, dtype=torch.int32)
    nodes[0, :3] = torch.tensor([1, 4, 30])
    nodes[4, :2] = torch.tensor([0, 18])
    p.lens = [3, 5, 8, 16, 2]
    p.dlens = torch.tensor(p.lens, dtype=torch.int32, device="cuda")
    p.table[1, 1] = p.table[1, 0]
    p.dtable = p.table.cuda()
    r = check_write(p, k, v, [3, 0, 0, 1, 2], nodes, bad=(0, 3))  # request 3's path holds a -1
    assert r["row_status"].tolist() == [B_.ROW_BAD_NODE, 0, 0, B_.ROW_BAD_NODE, 0]


def test_write_then_read_round_trip():
    g = torch.Generator().manual_seed(15)
    p = Pool(g, [0, 0], 4, 64, 128, spare=150)
    k, v = (torch.randn(2, 150, 4, 128, generator=g).cuda() for _ in range(2))
    r = sv.kv_cache_write(k, v, p.cache, p.dtable, p.dlens)
    back = sv.kv_cache_read(p.cache, p.dtable, r["lens"], max_len=150, dtype=torch.float32)
    for x, y, s in ((k, back["k"], p.cache.k_scale), (v, back["v"], p.cache.v_scale)):
        # half a step of e4m3, or half the smallest subnormal at the largest scale
        lim = 2.0 ** -4 * x.abs() + 2.0 ** -10 * float(s.nan_to_num().max())
        assert bool(((x - y).abs() <= lim).all())


# ------------------------------------------------------------------ attention

def run_attention(p, q, kn, vn, parents=None, n_rows=None, scale=None):
    B, T, hq, D = q.shape
    gd = Guarded()
    out = dict(out=gd.empty(q.shape, q.dtype, "out"), lse=gd.empty((B, T, hq), torch.float32, "lse"),
               row_status=gd.empty((B,), torch.int32, "status"))

    class Ws:
        def get(self, n):
            return gd.empty((n,), torch.uint8, "workspace")

    c = lambda x: None if x is None else x.cuda()
    sv.verify_attention(c(q), p.cache, p.dtable, p.dlens, k=c(kn), v=c(vn), parents=c(parents), n_rows=c(n_rows),
                        scale=scale, out=out, workspace=Ws())
    torch.cuda.synchronize()
    gd.check()
    return {k: v.cpu() for k, v in out.items()}


def check_attention(p, q, kn, vn, parents=None, n_rows=None, scale=None, skip=()):
    r = run_attention(p, q, kn, vn, parents, n_rows, scale)
    B, T, hq, D = q.shape
    s = D ** -0.5 if scale is None else scale
    for b in range(B):
        if b in skip:
            continue
        assert int(r["row_status"][b]) == 0
        kc, vc = p.line(0, b), p.line(1, b)
        live = T if n_rows is None else int(n_rows[b])
        ref = R.attention_ref(q[b], kc, vc, None if kn is None else kn[b], None if vn is None else vn[b],
                              None if parents is None else parents[b], live, s)
        out, lse, absv, seen, size = ref
        vmax = max([float(x.abs().max()) for x in (vc, torch.zeros(1) if vn is None else vn[b].double()) if x.numel()])
        tol, tl = R.attention_tolerance(out, lse, absv, seen, size, vmax, D, q.dtype)
        err = (r["out"][b].double() - out).abs()
        assert bool((err <= tol).all()), (b, float((err / tol.clamp(min=1e-300)).max()))
        got = r["lse"][b].double()
        assert bool((torch.isinf(got) == torch.isinf(lse)).all())
        fin = ~torch.isinf(lse)
        assert bool(((got - lse).abs()[fin] <= tl[fin]).all()), (b, float((got - lse).abs()[fin].max()))
    return r


def round_inputs(g, B, T, hq, hkv, D, dtype):
    q = (1.5 * torch.randn(B, T, hq, D, generator=g)).to(DT[dtype])
    kn, vn = (torch.randn(B, T, hkv, D, generator=g).to(DT[dtype]) for _ in range(2))
    return q, kn, vn


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("page,D,hq,hkv,T", [
    (16, 64, 2, 1, 1), (64, 128, 8, 8, 1), (32, 128, 8, 1, 2), (64, 128, 20, 4, 5), (16, 128, 16, 2, 6),
    (128, 64, 14, 2, 9), (64, 64, 8, 2, 17), (16, 128, 8, 1, 33)])
def test_attention_chain(dtype, page, D, hq, hkv, T):
    g = torch.Generator().manual_seed(page + D + hq + T)
    p = Pool(g, [0, 1, page - 1, page, 200, 777], hkv, page, D)
    q, kn, vn = round_inputs(g, 6, T, hq, hkv, D, dtype)
    check_attention(p, q, kn, vn)


@pytest.mark.parametrize("T,hq,hkv,D", [(2, 4, 1, 128), (17, 8, 2, 64), (65, 8, 2, 128), (130, 4, 2, 64), (256, 2, 1, 128)])
def test_attention_tree(T, hq, hkv, D):
    g = torch.Generator().manual_seed(T)
    p = Pool(g, [0, 5, 300], hkv, 32, D)
    q, kn, vn = round_inputs(g, 3, T, hq, hkv, D, "bf16")
    parents = torch.stack([R.random_parents(g, T - 1) for _ in range(3)])
    check_attention(p, q, kn, vn, parents)


@pytest.mark.parametrize("T,hq,hkv,D", [(130, 2, 1, 64), (140, 1, 1, 128), (256, 1, 1, 64)])
def test_attention_many_rows_tiles_follow_each_other(T, hq, hkv, D):
    # so many requests that one CTA takes all tiles of a request's own rows, and the next request's after them
    g = torch.Generator().manual_seed(T)
    lens = [0, 0, 0, 40] * 30
    p = Pool(g, lens, hkv, 32, D)
    q, kn, vn = round_inputs(g, len(lens), T, hq, hkv, D, "bf16")
    parents = torch.stack([R.random_parents(g, T - 1) for _ in lens])
    check_attention(p, q, kn, vn, parents)
    check_attention(p, q, kn, vn)


@pytest.mark.parametrize("T,hq,hkv", [(1, 1, 1), (1, 32, 8), (4, 32, 4), (9, 16, 2)])
def test_attention_long_context(T, hq, hkv):
    """Long and ragged contexts: parts of many CTAs are joined."""
    g = torch.Generator().manual_seed(T + hq)
    p = Pool(g, [9001, 3, 4097], hkv, 64, 128)
    q, kn, vn = round_inputs(g, 3, T, hq, hkv, 128, "bf16")
    check_attention(p, q, kn, vn)


def test_attention_many_requests():
    g = torch.Generator().manual_seed(77)
    lens = [int(x) for x in torch.randint(0, 90, (131,), generator=g)]
    p = Pool(g, lens, 2, 16, 64)
    q, kn, vn = round_inputs(g, 131, 3, 4, 2, 64, "bf16")
    check_attention(p, q, kn, vn)


@pytest.mark.parametrize("T", [1, 40])
def test_attention_cache_alone_and_dead_rows(T):
    g = torch.Generator().manual_seed(21)
    p = Pool(g, [0, 17, 130, 64], 2, 16, 128)
    q, kn, vn = round_inputs(g, 4, T, 8, 2, 128, "f16")
    r = check_attention(p, q, None, None)
    assert bool((r["out"][0] == 0).all()) and bool(torch.isneginf(r["lse"][0]).all())
    n_rows = torch.tensor([0, T, max(1, T // 2), 0], dtype=torch.int32)
    check_attention(p, q, kn, vn, n_rows=n_rows)


def test_attention_unseen_values_have_no_effect():
    """NaN and infinities in rows that a row does not see, and in slots past the length (Pool fills those with NaN)."""
    g = torch.Generator().manual_seed(22)
    T = 12
    p = Pool(g, [0, 33], 2, 16, 64)
    q, kn, vn = round_inputs(g, 2, T, 8, 2, 64, "bf16")
    parents = torch.full((2, T - 1), -1, dtype=torch.int32)  # every node a child of the frontier
    clean = run_attention(p, q, kn, vn, parents)
    k2, v2 = kn.clone(), vn.clone()
    k2[:, 5], v2[:, 5] = math.nan, math.inf
    v2[:, 7, 0, 3] = math.nan
    k2[:, 9, 1] = -math.inf
    r = run_attention(p, q, k2, v2, parents)
    for t in range(T):
        if t not in (5, 7, 9):
            assert torch.equal(r["out"][:, t], clean["out"][:, t]) and torch.equal(r["lse"][:, t], clean["lse"][:, t])
    assert bool(r["out"][:, 5].isnan().all())
    assert bool(r["out"][:, 7, :4, 3].isnan().all()) and not bool(r["out"][:, 7, :, 4:].isnan().any())
    # a NaN in the cache reaches every row of its head
    p.cache.v.view(torch.uint8)[int(p.table[1, 1]), 1, 2, 9] = 0x7F
    r = run_attention(p, q, kn, vn, parents)
    assert bool(r["out"][1, :, 4:, 9].isnan().all()) and not bool(r["out"][1, :, :4].isnan().any())
    assert not bool(r["out"][0].isnan().any())
    # a row of q that is not finite gives NaN, the others stay
    q2 = q.clone()
    q2[1, 2, 3, 0] = math.inf
    r = run_attention(p, q2, kn, vn, parents)
    assert bool(r["out"][1, 2, 3].isnan().all()) and not bool(r["out"][1, 3].isnan().all())


def test_attention_extreme_scores_and_scales():
    """Scores far apart, and pages whose scales differ by 2^40: the largest scale is not the heaviest page."""
    g = torch.Generator().manual_seed(23)
    p = Pool(g, [200, 64], 1, 16, 64)
    for b in range(2):
        for j in range(p.lens[b] // 16):
            page = int(p.table[b, j])
            p.scales[1][page] = 2.0 ** (-30 + 10 * (j % 5))
    p.cache.v_scale.copy_(p.scales[1])
    q, kn, vn = round_inputs(g, 2, 3, 4, 1, 64, "bf16")
    q[0] *= 30
    check_attention(p, q, kn, vn)


def test_attention_bad_requests():
    g = torch.Generator().manual_seed(24)
    p = Pool(g, [300, 40, 64, 10], 2, 16, 128)
    T = 5
    q, kn, vn = round_inputs(g, 4, T, 8, 2, 128, "bf16")
    p.dtable[0, 11] = -1
    p.dlens[2] = 10 ** 6
    parents = torch.stack([R.random_parents(g, T - 1) for _ in range(4)])
    parents[3, 2] = 2
    r = check_attention(p, q, kn, vn, parents, skip=(0, 2, 3))
    assert r["row_status"].tolist() == [B_.ROW_BAD_PAGE, 0, B_.ROW_BAD_LENGTH, B_.ROW_BAD_PARENT]
    for b in (0, 2, 3):
        assert bool(r["out"][b].isnan().all()) and bool(r["lse"][b].isnan().all())


def test_attention_strided_inputs_and_streams():
    g = torch.Generator().manual_seed(25)
    p = Pool(g, [100, 3], 2, 32, 128)
    qkv = torch.randn(2, 4, (8 + 2 + 2) * 128 + 1, generator=g).bfloat16()
    q = qkv[..., 1:1 + 1024].unflatten(-1, (8, 128))
    kn = qkv[..., 1025:1025 + 256].unflatten(-1, (2, 128))
    vn = qkv[..., 1281:1281 + 256].unflatten(-1, (2, 128))
    check_attention(p, q, kn, vn)
    dev = qkv.cuda()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    args = [dev[..., 1:1025].unflatten(-1, (8, 128)), p.cache, p.dtable, p.dlens]
    kw = dict(k=dev[..., 1025:1281].unflatten(-1, (2, 128)), v=dev[..., 1281:1537].unflatten(-1, (2, 128)), lse=True)
    a = sv.verify_attention(*args, **kw)
    b = sv.verify_attention(*args, stream=st, **kw)
    torch.cuda.synchronize()
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def test_attention_is_deterministic_and_captures():
    g = torch.Generator().manual_seed(26)
    p = Pool(g, [5000, 100], 2, 64, 128)
    q, kn, vn = (x.cuda() for x in round_inputs(g, 2, 6, 16, 2, 128, "bf16"))
    ws = sv.Workspace()
    call = lambda: sv.verify_attention(q, p.cache, p.dtable, p.dlens, k=kn, v=vn, lse=True, workspace=ws)
    a = call()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c = call()
    for _ in range(3):
        c["out"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a["out"], c["out"]) and torch.equal(a["lse"], c["lse"])


# ------------------------------------------------------------------ logits

def logits_case(seed, B, Rr, V, H, nb, dtype, tree, mask):
    g = torch.Generator().manual_seed(seed)
    N = Rr - 1
    c = dict(logits=(3 * torch.randn(B, Rr, V, generator=g)).to(DT[dtype]))
    lo = max(1, V // 10)
    c["history"] = torch.randint(0, lo, (B, H), generator=g, dtype=torch.int32)
    c["history"][:, ::7] = -1                       # padding
    c["history"][:, 3::11] = V
    c["tokens"] = torch.randint(0, lo, (B, N), generator=g, dtype=torch.int32)
    if N > 3:
        c["tokens"][:, 3] = c["tokens"][:, 0]
    c["history_len"] = torch.randint(0, H + 1, (B,), generator=g, dtype=torch.int32)
    c["prompt_len"] = (c["history_len"] // 2).to(torch.int32)
    c["parents"] = torch.stack([R.random_parents(g, N) for _ in range(B)]) if tree and N else None
    for n, lo_, hi in (("repetition", 0.8, 1.5), ("presence", -0.5, 1.0), ("frequency", -0.2, 0.7)):
        c[n] = lo_ + (hi - lo_) * torch.rand(B, generator=g)
    c["bias_tokens"] = c["bias_values"] = c["allowed"] = None
    if nb:
        c["bias_tokens"] = torch.randint(-1, V + 1, (B, nb), generator=g, dtype=torch.int32)
        c["bias_values"] = 4 * torch.randn(B, nb, generator=g)
    if mask:
        c["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (B, Rr, (V + 31) // 32), generator=g, dtype=torch.int64).to(torch.int32)
    return c


def check_logits(c, in_place=False, logits=None):
    dev = {k: None if x is None else x.cuda() for k, x in c.items()}
    if logits is not None:
        dev["logits"] = logits
    x = dev.pop("logits")
    if not c["tokens"].shape[1]:
        dev["tokens"] = None
    gd = Guarded()
    out = dict(logits=x if in_place else gd.empty(c["logits"].shape, x.dtype, "out"),
               row_status=gd.empty((x.shape[0],), torch.int32, "status"))
    sv.process_logits(x, out=out, **dev)
    torch.cuda.synchronize()
    gd.check()
    B, Rr, V = c["logits"].shape
    got = out["logits"].cpu()
    half = torch.finfo(got.dtype).eps / 2
    for b in range(B):
        for r in range(Rr):
            allowed = None
            if c["allowed"] is not None:
                w = c["allowed"][b, r].long()
                allowed = ((w[:, None] >> torch.arange(32)) & 1).flatten()[:V].bool()
            bias = [] if c["bias_tokens"] is None else list(zip(c["bias_tokens"][b].tolist(), c["bias_values"][b].double().tolist()))
            f = lambda n: float(c[n][b])
            want = R.logits_ref(c["logits"][b, r], r, c["tokens"][b], None if c["parents"] is None else c["parents"][b],
                                c["history"][b], int(c["prompt_len"][b]), int(c["history_len"][b]), f("repetition"),
                                f("presence"), f("frequency"), bias, allowed)
            y = got[b, r].double()
            inf = torch.isinf(want)
            assert bool((torch.isinf(y) == inf).all())
            # at most five fp32 roundings of magnitudes up to the terms', then the type's own
            big = c["logits"][b, r].double().abs() * 2 + 0.7 * 1.1 * c["history"].shape[1] + 20
            tol = 5 * 2.0 ** -24 * big + half * want.abs()
            assert bool(((y - want).abs()[~inf] <= tol[~inf]).all()), (b, r)
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Rr,V,H,nb,tree,mask", [
    (1, 1, 1, 1, 0, False, False), (2, 1, 37, 20, 3, False, True), (3, 6, 4096, 300, 10, False, False),
    (2, 9, 5003, 100, 0, True, True), (2, 65, 8200, 500, 40, True, True), (1, 5, 50000, 1000, 300, False, False)])
def test_logits(dtype, B, Rr, V, H, nb, tree, mask):
    out = check_logits(logits_case(V + Rr, B, Rr, V, H, nb, dtype, tree, mask))
    assert out["row_status"].tolist() == [0] * B


def test_logits_in_place_and_strided():
    c = logits_case(3, 3, 5, 1000, 64, 5, "bf16", True, True)
    check_logits(c, in_place=True, logits=c["logits"].cuda())
    big = torch.zeros(3, 5, 1001, dtype=torch.bfloat16, device="cuda")
    big[..., 1:] = c["logits"].cuda()
    check_logits(c, logits=big[..., 1:])
    check_logits(c, in_place=True, logits=big[..., 1:])


def test_logits_special_values_and_defaults():
    x = torch.tensor([[[1.0, -2.0, math.nan, math.inf, -math.inf, 0.0, -0.0, 5.0]]]).cuda()
    r = sv.process_logits(x)["logits"]
    assert same(r.cpu(), x.cpu())
    hist = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    two = torch.tensor([2.0], device="cuda")
    r = sv.process_logits(x, history=hist, repetition=two)["logits"][0, 0].cpu()
    assert r.tolist()[:2] == [0.5, -4.0] and math.isnan(r[2]) and r[3] == math.inf and r[4] == -math.inf and r[7] == 2.5
    # a mask of no token, and a NaN under the mask
    none = torch.zeros(1, 1, 1, dtype=torch.int32, device="cuda")
    assert bool(torch.isneginf(sv.process_logits(x, allowed=none)["logits"]).all())


def test_logits_bad_parent():
    c = logits_case(4, 3, 6, 500, 30, 0, "f32", True, False)
    c["parents"][1, 3] = 3
    c["parents"][2, 0] = -2
    out = check_logits(c)
    assert out["row_status"].tolist() == [0, B_.ROW_BAD_PARENT, B_.ROW_BAD_PARENT]


# ------------------------------------------------------------------ waits and the whole round

def test_attention_wait_limit_reports_a_timeout():
    """With no polls allowed every wait of the many-rows kernel runs out at once: status and NaN, no hang; afterwards the
    same call gives what it gave before."""
    g = torch.Generator().manual_seed(31)
    p = Pool(g, [700, 3, 0], 2, 64, 128)
    q, kn, vn = round_inputs(g, 3, 6, 8, 2, 128, "bf16")
    clean = run_attention(p, q, kn, vn)
    old = sv.set_wait_limit(0)
    try:
        r = run_attention(p, q, kn, vn)
    finally:
        sv.set_wait_limit(old)
    assert r["row_status"].tolist() == [B_.ROW_TIMEOUT] * 3
    assert bool(r["out"].isnan().all()) and bool(r["lse"].isnan().all())
    again = run_attention(p, q, kn, vn)
    assert torch.equal(again["out"], clean["out"]) and torch.equal(again["lse"], clean["lse"])


@pytest.mark.parametrize("T,hq,hkv,dtype", [(24, 16, 1, "bf16"), (40, 16, 1, "f16"), (65, 16, 1, "bf16"), (17, 1, 1, "f16"), (128, 2, 1, "bf16")])
def test_attention_many_rows_of_a_head(T, hq, hkv, dtype):
    """Rows that fill several row tiles, with an odd rest."""
    g = torch.Generator().manual_seed(T * hq)
    p = Pool(g, [129, 1000], hkv, 128, 128)
    q, kn, vn = round_inputs(g, 2, T, hq, hkv, 128, dtype)
    check_attention(p, q, kn, vn)


@pytest.mark.parametrize("hq,T", [(1, 1), (8, 5)])
def test_attention_reference_moves_late(hq, T):
    """Scores that climb along the context, so that the running maximum leaves its window again and again."""
    g = torch.Generator().manual_seed(33)
    p = Pool(g, [2000], 1, 16, 64)
    q, kn, vn = round_inputs(g, 1, T, hq, 1, 64, "bf16")
    q[:] = q.abs() + 0.5
    for j in range(125):
        page = int(p.table[0, j])
        p.codes[0][page] = torch.full((1, 16, 64), 1.0 + 0.0625 * (j % 8)).to(R.FP8)
        p.scales[0][page] = 2.0 ** (-6 + j // 16)
    p.cache.k.view(torch.uint8).copy_(p.codes[0].view(torch.uint8).cuda())
    p.cache.k_scale.copy_(p.scales[0])
    check_attention(p, q, kn, vn)


@pytest.mark.parametrize("tree", [False, True])
def test_example_runs_a_whole_round(tree):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verification_round.py")
    spec = importlib.util.spec_from_file_location("verification_round", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    r = ex.run(rounds=3, tree=tree)
    acc = r["accepted"]
    assert bool((acc >= 0).all())
    if tree:
        assert int(acc.sum()) > 0
    assert r["lens"].tolist() == (149 + (acc + 1).sum(0)).tolist()
    assert r["hist_len"].tolist() == (r["lens"] + 1).tolist()
    # what the cache holds are the keys of the committed tokens, to a code's precision
    toy = r["toy"]
    for b in range(acc.shape[1]):
        n = int(r["lens"][b])
        _, _, k, _ = toy.qkv(r["history"][b, :n])
        got, want = r["cache_k"][b, :n], k.float()
        lim = 2.0 ** -4 * want.abs() + 2.0 ** -10 * (2 * want.abs().max() / 448 * 2)
        assert bool(((got - want).abs() <= lim).all())


@pytest.mark.parametrize("hq,T", [(2, 4), (8, 9)])
def test_attention_keys_that_are_not_finite(hq, T):
    """A key of the round with an infinity gives NaN to the rows that see it and to no other, on both paths."""
    g = torch.Generator().manual_seed(35)
    p = Pool(g, [0, 40], 1, 16, 128)
    q, kn, vn = round_inputs(g, 2, T, hq, 1, 128, "bf16")
    clean = run_attention(p, q, kn, vn)
    kn[:, 2, 0, 7] = -math.inf
    r = run_attention(p, q, kn, vn)
    assert bool(r["out"][:, 2:].isnan().all()) and bool(r["lse"][:, 2:].isnan().all())
    assert torch.equal(r["out"][:, :2], clean["out"][:, :2]) and torch.equal(r["lse"][:, :2], clean["lse"][:, :2])
