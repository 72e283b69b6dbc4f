"""The calls around the verify step where they can go wrong: scores past 2^24, waits that run out in one CTA, long prompts,
streams, captures, and both attention kernels (T Hq / Hkv up to 16 rows, and more) on the same inputs."""
import math

import pytest
import torch

import speculative_decoding_verification_spec_gb300 as sv
from speculative_decoding_verification_spec_gb300 import binding as B_

import round_ref as R
from test_gpu_round import DT, Pool, check_attention, check_write, round_inputs, run_attention, same

pytestmark = pytest.mark.gpu


def copies(p, n):
    """The pool's requests n times over (they share their pages), so that a CTA works through a request's tiles one after another."""
    p.dtable, p.dlens = p.dtable.repeat(n, 1), p.dlens.repeat(n)


# ------------------------------------------------------------------ both kernels, T hq / hkv up to 16 and more

@pytest.mark.parametrize("T,hq", [(3, 4), (9, 8)])
def test_attention_without_rows_of_the_round_has_no_use_for_parents(T, hq):
    g = torch.Generator().manual_seed(40)
    p = Pool(g, [0, 40], 2, 16, 64)
    q, _, _ = round_inputs(g, 2, T, hq, 2, 64, "bf16")
    want = run_attention(p, q, None, None)
    r = run_attention(p, q, None, None, parents=torch.full((2, T - 1), 9, dtype=torch.int32))
    assert r["row_status"].tolist() == [0, 0]
    assert all(torch.equal(r[n], want[n]) for n in r)


BOTH = [(1, 8, 2), (3, 8, 2), (5, 8, 2), (9, 16, 2)]


@pytest.mark.parametrize("T,hq,hkv", BOTH)
def test_attention_bad_requests_on_both_paths(T, hq, hkv):
    """A bad page in the middle and at the end of a context whose parts are joined, a bad length, a bad parent."""
    g = torch.Generator().manual_seed(44)
    lens = [9001, 40, 64, 10, 4097, 9001]
    p = Pool(g, lens, hkv, 16, 128)
    q, kn, vn = round_inputs(g, len(lens), T, hq, hkv, 128, "bf16")
    p.dtable[0, 300] = -1
    p.dtable[4, 256] = p.codes[0].shape[0]
    p.dlens[2] = -1
    bad = {0: B_.ROW_BAD_PAGE, 2: B_.ROW_BAD_LENGTH, 4: B_.ROW_BAD_PAGE}
    parents = None
    if T > 2:
        parents = torch.stack([R.random_parents(g, T - 1) for _ in lens])
        parents[3, T - 2] = T - 2
        parents[5, 1] = -2
        bad.update({3: B_.ROW_BAD_PARENT, 5: B_.ROW_BAD_PARENT})
    r = check_attention(p, q, kn, vn, parents, skip=tuple(bad))
    assert r["row_status"].tolist() == [bad.get(b, 0) for b in range(len(lens))]
    for b in bad:
        assert bool(r["out"][b].isnan().all()) and bool(r["lse"][b].isnan().all())


@pytest.mark.parametrize("lens", [[0, 33], [5000, 9]])
@pytest.mark.parametrize("T,hq", [(8, 4), (8, 8)])
def test_attention_unseen_values_on_both_paths(T, hq, lens):
    """NaN and infinities in rows that a row does not see, in the cache and in q."""
    g = torch.Generator().manual_seed(45)
    p = Pool(g, lens, 2, 16, 64)
    q, kn, vn = round_inputs(g, 2, T, hq, 2, 64, "bf16")
    parents = torch.full((2, T - 1), -1, dtype=torch.int32)  # every node a child of the frontier
    clean = run_attention(p, q, kn, vn, parents)
    k2, v2 = kn.clone(), vn.clone()
    k2[:, 3], v2[:, 3] = math.nan, math.inf
    v2[:, 5, 0, 3] = math.nan
    v2[:, 6, 1, 60] = -math.inf
    r = run_attention(p, q, k2, v2, parents)
    for t in range(T):
        if t not in (3, 5, 6):
            assert torch.equal(r["out"][:, t], clean["out"][:, t]) and torch.equal(r["lse"][:, t], clean["lse"][:, t])
    G = hq // 2
    assert bool(r["out"][:, 3].isnan().all()) and bool(r["lse"][:, 3].isnan().all())
    assert bool(r["out"][:, 5, :G, 3].isnan().all()) and torch.equal(r["out"][:, 5, G:], clean["out"][:, 5, G:])
    assert bool(torch.isneginf(r["out"][:, 6, G:, 60]).all()) and torch.equal(r["out"][:, 6, :G], clean["out"][:, 6, :G])
    b = lens.index(min(x for x in lens if x > 0))
    p.cache.v.view(torch.uint8)[int(p.table[b, 0]), 1, 2, 9] = 0x7F
    r = run_attention(p, q, kn, vn, parents)
    assert bool(r["out"][b, :, G:, 9].isnan().all()) and not bool(r["out"][b, :, :G].isnan().any())
    assert torch.equal(r["out"][1 - b], clean["out"][1 - b])
    q2 = q.clone()
    q2[1, 2, 1, 0] = math.inf
    q2[0, 1, 0, 7] = math.nan
    p.cache.v.view(torch.uint8)[int(p.table[b, 0]), 1, 2, 9] = 0
    p.codes[1].view(torch.uint8)[int(p.table[b, 0]), 1, 2, 9] = 0
    r, want = run_attention(p, q2, kn, vn, parents), run_attention(p, q, kn, vn, parents)
    assert bool(r["out"][1, 2, 1].isnan().all()) and bool(r["out"][0, 1, 0].isnan().all())
    gone = r["lse"].isnan()
    assert int(gone.sum()) == 2 and torch.equal(r["out"][~gone], want["out"][~gone])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,hq,hkv,D", [(2, 8, 2, 64), (9, 8, 2, 64), (9, 8, 2, 128), (70, 4, 1, 128)])
def test_attention_unaligned_rows_on_both_paths(T, hq, hkv, D, dtype):
    """q, k and v cut out of one buffer at odd offsets, with row strides that allow no wide load."""
    g = torch.Generator().manual_seed(46)
    p = Pool(g, [100, 3], hkv, 32, D)
    qkv = torch.randn(2, T, (hq + 2 * hkv) * D + 3, generator=g).to(DT[dtype]).cuda()
    cut = lambda at, h: qkv[..., at:at + h * D].unflatten(-1, (h, D))
    q, kn, vn = cut(1, hq), cut(1 + hq * D, hkv), cut(3 + (hq + hkv) * D, hkv)
    assert not q.is_contiguous() and q.data_ptr() % 4 and vn.data_ptr() % 4
    check_attention(p, q.cpu(), kn.cpu(), vn.cpu())
    dense = sv.verify_attention(q.contiguous(), p.cache, p.dtable, p.dlens, k=kn.contiguous(), v=vn.contiguous(), lse=True)
    r = sv.verify_attention(q, p.cache, p.dtable, p.dlens, k=kn, v=vn, lse=True)
    assert all(torch.equal(r[n], dense[n]) for n in r)
    # heads before rows, and one batch stride for all
    qt, kt, vt = (x.contiguous().transpose(1, 2).contiguous().transpose(1, 2) for x in (q, kn, vn))
    r = sv.verify_attention(qt, p.cache, p.dtable, p.dlens, k=kt, v=vt, lse=True)
    assert all(torch.equal(r[n], dense[n]) for n in r)
    one = [x[:1].expand(2, *x.shape[1:]) for x in (q, kn, vn)]
    r = sv.verify_attention(one[0], p.cache, p.dtable, p.dlens, k=one[1], v=one[2], lse=True)
    assert all(torch.equal(r[n][0], dense[n][0]) for n in ("out", "lse"))


@pytest.mark.parametrize("T,hq,hkv,D", [(4, 8, 2, 64), (17, 8, 2, 64), (65, 8, 2, 128), (130, 4, 2, 64)])
def test_attention_tree_f16(T, hq, hkv, D):
    g = torch.Generator().manual_seed(T)
    p = Pool(g, [0, 5, 300], hkv, 32, D)
    q, kn, vn = round_inputs(g, 3, T, hq, hkv, D, "f16")
    parents = torch.stack([R.random_parents(g, T - 1) for _ in range(3)])
    check_attention(p, q, kn, vn, parents)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,hq", [(3, 4), (9, 4), (20, 6)])
def test_attention_scales_far_apart(T, hq, dtype):
    """Pages whose values differ by 2^40 in scale, the heavy tokens on those with the smallest: what a weight may be off by is counted
    against the largest p 2^e of the row, not against the largest value."""
    g = torch.Generator().manual_seed(47)
    D, page, n = 64, 16, 640
    p = Pool(g, [n], 1, page, D)
    e = torch.zeros(n)
    for j in range(n // page):
        i = int(p.table[0, j])
        p.scales[1][i] = 2.0 ** (-30 + 10 * (j % 5))
        p.scales[0][i] = 2.0 ** (-4 if j % 5 == 0 else -6)
        e[j * page:(j + 1) * page] = -30 + 10 * (j % 5)
    p.cache.k_scale.copy_(p.scales[0])
    p.cache.v_scale.copy_(p.scales[1])
    q, _, _ = round_inputs(g, 1, T, hq, 1, D, dtype)
    copies(p, 320)
    r = run_attention(p, q.repeat(320, 1, 1, 1), None, None)
    kc, vc = p.line(0, 0), p.line(1, 0)
    out, lse, absv, seen, size = R.attention_ref(q[0], kc, vc, None, None, None, T, D ** -0.5)
    w = torch.exp(torch.einsum("thd,jd->thj", q[0].double(), kc[:, 0]) * D ** -0.5 - lse[..., None])
    top = (w * torch.exp2(e.double())).amax(-1, keepdim=True)
    tol, tl = R.attention_tolerance(out, lse, absv, seen, size, 0.0, D, q.dtype)
    tol = tol + n * 2.0 ** -32 * top * 448
    if dtype == "f16":
        assert float(out.abs().max()) < 60000
    for b in range(320):
        err = (r["out"][b].double() - out).abs()
        assert bool((err <= tol).all()), (b, float((err / tol).max()))
        assert bool(((r["lse"][b].double() - lse).abs() <= tl).all()), b


# ------------------------------------------------------------------ waits that run out

@pytest.mark.parametrize("T,hq,hkv,lens", [(6, 16, 4, [900, 3, 0, 2100]), (40, 8, 8, [600] * 24), (6, 32, 8, [70] * 90)])
def test_attention_time_outs_of_any_head_are_reported(T, hq, hkv, lens):
    """Limits under which waits run out in some CTAs and not in others: a request without a status holds what it held before, and one
    with the status holds nothing else but NaN."""
    g = torch.Generator().manual_seed(51)
    p = Pool(g, lens, hkv, 64, 128)
    q, kn, vn = (x.cuda() for x in round_inputs(g, len(lens), T, hq, hkv, 128, "bf16"))
    call = lambda: sv.verify_attention(q, p.cache, p.dtable, p.dlens, k=kn, v=vn, lse=True)
    clean = call()
    seen = set()
    for limit in [1, 2, 3, 4, 6, 8, 12] * 12:
        old = sv.set_wait_limit(limit)
        try:
            r = call()
        finally:
            sv.set_wait_limit(old)
        status = r["row_status"].tolist()
        seen.update(status)
        for name in ("out", "lse"):
            x, y = r[name].flatten(1), clean[name].flatten(1)
            gone = x.isnan()
            assert bool(((x == y) | gone).all()), (limit, name)
            lost = gone.any(1).tolist()
            assert all(s == B_.ROW_TIMEOUT for s, l in zip(status, lost) if l), (limit, name, status, lost)
    assert seen <= {B_.ROW_OK, B_.ROW_TIMEOUT}
    again = call()
    assert torch.equal(again["out"], clean["out"]) and torch.equal(again["lse"], clean["lse"])


# ------------------------------------------------------------------ scores past 2^24

def in_hull(out, v):
    """Whether every output lies between the least and the largest value of its head, to its type's rounding."""
    lo, hi = v.amin(0), v.amax(0)  # [heads, D]
    room = 2.0 ** -10 * torch.maximum(lo.abs(), hi.abs())
    G = out.shape[1] // v.shape[1]
    lo, hi, room = (x.repeat_interleave(G, 0) for x in (lo, hi, room))
    return bool(((out >= lo - room) & (out <= hi + room)).all())


@pytest.mark.parametrize("later,ve", [(1.0, (-8, -8)), (0.0, (-12, 0)), (0.0, (-8, 8)), (0.0, (8, -40))])
@pytest.mark.parametrize("T,hq", [(2, 4), (6, 16)])
def test_attention_neighbouring_scores_past_2_27(T, hq, later, ve):
    """Scores (or their sums with the values' exponents) that are neighbouring floats, 16 apart, with the larger ones later: the
    reference cannot lie between them."""
    g = torch.Generator().manual_seed(41)
    D, page, n = 128, 64, 512
    p = Pool(g, [n], 1, page, D)
    for j in range(n // page):
        k = torch.full((1, page, D), 1.5)
        late = j >= n // page // 2
        k[..., -1] = later if late else 0.0
        i = int(p.table[0, j])
        p.codes[0][i] = k.to(R.FP8)
        p.scales[0][i] = 1.0
        p.scales[1][i] = 2.0 ** ve[late]
    p.cache.k.view(torch.uint8).copy_(p.codes[0].view(torch.uint8).cuda())
    p.cache.k_scale.copy_(p.scales[0])
    p.cache.v_scale.copy_(p.scales[1])
    q = torch.full((1, T, hq, D), 2.0 ** 20)
    q[..., -1] = 2.0 ** 4                      # log2(e) s = 190.5 2^20, and 16 more
    more = torch.exp2(torch.arange(T * hq) % 4.0).view(T, hq)
    q = (q * more[None, ..., None]).bfloat16()
    copies(p, 320)
    r = run_attention(p, q.repeat(320, 1, 1, 1), None, None, scale=math.log(2.0))
    assert r["row_status"].tolist() == [0] * 320
    top = 190.5 * 2.0 ** 20 * more * math.log(2.0)
    for b in range(320):
        assert in_hull(r["out"][b].double(), p.line(1, 0)), b
        assert bool(((r["lse"][b] / top - 1).abs() <= 2.0 ** -20).all()), b


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,hq", [(1, 4), (3, 5), (3, 8), (9, 16)])
@pytest.mark.parametrize("e", [11, 16, 17, 18, 19, 22, 30, 60])
def test_attention_huge_scores(T, hq, dtype, e):
    """|log2(e) s| from 2^20 to 2^70, values of pages with several exponents: every tile is left after one repeat, and where one token
    stands clear of the scores' own rounding the output is its value."""
    g = torch.Generator().manual_seed(100 * T + e)
    D = 128
    p = Pool(g, [700, 130], 1, 16, D)
    p.codes[0] = p.codes[0].float().abs().to(R.FP8)
    p.scales[0][:] = 2.0 ** e
    p.cache.k.view(torch.uint8).copy_(p.codes[0].view(torch.uint8).cuda())
    p.cache.k_scale.copy_(p.scales[0])
    q, kn, vn = round_inputs(g, 2, T, hq, 1, D, dtype)
    q = (q.abs() + 0.5).to(DT[dtype])
    n = 160
    copies(p, n)
    r = run_attention(p, *(x.repeat(n, 1, 1, 1) for x in (q, kn, vn)))
    assert r["row_status"].tolist() == [0] * (2 * n)
    clear = 0
    for b in range(2):
        kc, vc = p.line(0, b), p.line(1, b)
        out, lse, absv, seen, size = R.attention_ref(q[b], kc, vc, kn[b], vn[b], None, T, D ** -0.5)
        vmax = float(max(vc.abs().max(), vn.abs().max()))
        tol, _ = R.attention_tolerance(out, lse, absv, seen, torch.zeros_like(size), vmax, D, q.dtype)
        ds = D * 2.0 ** -23 * size
        s = torch.einsum("thd,jd->thj", q[b].double(), kc[:, 0]) * D ** -0.5
        best = s.topk(2).values
        ok = best[..., 0] - best[..., 1] > 4 * ds + 64
        clear += int(ok.sum())
        for c in range(b, 2 * n, 2):
            assert in_hull(r["out"][c].double(), torch.cat([vc, vn[b].double()])), c
            assert bool(((r["lse"][c].double() - lse).abs() <= 2 * ds + 2.0 ** -22 * lse.abs() + 1e-3).all()), c
            assert bool(((r["out"][c].double() - out).abs() <= tol)[ok].all()), c
    assert clear >= T * hq


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,hq", [(1, 4), (4, 16)])
def test_attention_small_weights_beside_a_large_one(T, hq, dtype):
    """One token holds nearly all of the weight and a value near zero, 32767 others share the rest and make the output."""
    D, page, n = 128, 64, 32768
    g = torch.Generator().manual_seed(43)
    p = Pool(g, [n], 1, page, D)
    for which, (one, rest) in enumerate(((1.5, 0.125), (2.0 ** -9, 1.0))):
        p.codes[which] = torch.full(p.codes[which].shape, rest).to(R.FP8)
        p.codes[which][int(p.table[0, 0]), 0, 0] = torch.full((D,), one).to(R.FP8)
        p.scales[which].fill_(1.0)
        p.cache[which].view(torch.uint8).copy_(p.codes[which].view(torch.uint8).cuda())
        p.cache[2 + which].copy_(p.scales[which])
    q = (1.0 - 2.0 ** -8 * (torch.arange(T * hq) % 8).view(1, T, hq, 1)).expand(1, T, hq, D).to(DT[dtype])
    copies(p, 320)
    r = run_attention(p, q.repeat(320, 1, 1, 1), None, None)
    kc, vc = p.line(0, 0), p.line(1, 0)
    out, lse, absv, seen, size = R.attention_ref(q[0], kc, vc, None, None, None, T, D ** -0.5)
    assert float(out.max()) < 0.05 and bool((out > 0.003).all())
    # weights: 2^-11 of each, or 2^-32 of the largest; sums of n tokens, 16 a step, and two scores that fp32 holds but for their last
    # places: 2^-11; the output's own rounding
    tol = n * 2.0 ** -32 + (2 * 2.0 ** -11 + torch.finfo(q.dtype).eps / 2) * out
    for b in range(320):
        err = (r["out"][b].double() - out).abs()
        assert bool((err <= tol).all()), (b, float((err / out).max()), float((tol / out).min()))
        assert bool(((r["lse"][b].double() - lse).abs() <= 2.0 ** -14).all())


# ------------------------------------------------------------------ long prompts

@pytest.mark.parametrize("T,page,D,accepted", [(17000, 16, 64, [16999, 9001, -1]), (33000, 32, 128, None)])
def test_write_of_a_long_prompt(T, page, D, accepted):
    """More pages than a CTA's share: a CTA takes several."""
    g = torch.Generator().manual_seed(61)
    B = 3 if accepted else 1
    p = Pool(g, [0, page - 3, 2 * page][:B], 1, page, D, spare=T)
    mag = torch.exp2(torch.randint(-6, 7, (B, T, 1, 1), generator=g).float())
    k, v = ((torch.randn(B, T, 1, D, generator=g) * mag).bfloat16().cuda() for _ in range(2))
    check_write(p, k, v, accepted)


def test_write_of_a_long_prompt_refuses_it_whole():
    g = torch.Generator().manual_seed(62)
    T = 17000
    p = Pool(g, [5, 9], 1, 16, 64, spare=T)
    k, v = (torch.randn(2, T, 1, 64, generator=g).bfloat16().cuda() for _ in range(2))
    p.table[0, 1062] = p.codes[0].shape[0]
    p.dtable = p.table.cuda()
    r = check_write(p, k, v, bad=(0,))
    assert r["row_status"].tolist() == [B_.ROW_BAD_PAGE, 0]


def test_write_time_grows_with_the_tokens():
    """Four times the tokens take about four times as long, not sixteen."""
    def time(T):
        cache = sv.kv_cache(T // 16, 1, 16, 64)
        table = torch.randperm(T // 16, device="cuda").to(torch.int32)[None]
        lens = torch.zeros(1, dtype=torch.int32, device="cuda")
        k = torch.randn(1, T, 1, 64, device="cuda").bfloat16()
        out = sv.kv_cache_write(k, k, cache, table, lens)
        best = math.inf
        for _ in range(10):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            sv.kv_cache_write(k, k, cache, table, lens, out=out)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    assert time(1 << 19) < 7 * time(1 << 17)


def test_write_of_a_path_without_room_for_nodes():
    """A tree call with room for one token gives out_nodes of width 0: row 0 may be written, and nothing that a path would name."""
    g = torch.Generator().manual_seed(63)
    T = 4
    p = Pool(g, [3, 5, 17], 2, 16, 64, spare=T)
    k, v = (torch.randn(3, T, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    r = check_write(p, k, v, [0, 2, -1], torch.empty(3, 0, dtype=torch.int32), bad=(1,))
    assert r["row_status"].tolist() == [0, B_.ROW_BAD_LENGTH, 0]


# ------------------------------------------------------------------ streams and captures

def busy_block(nbytes, value):
    """A block that the caching allocator hands out next on the current stream, while that still has to write `value` to it."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(400_000_000)  # some 0.2 s
    x.fill_(value)
    return x.data_ptr()


@pytest.mark.parametrize("what", ["attention", "logits", "write", "read"])
def test_new_outputs_on_another_stream_are_the_calls_own(what):
    """The current stream still has work on a block that was freed there; a call on another stream does not take it."""
    g = torch.Generator().manual_seed(71)
    p = Pool(g, [70, 130], 2, 32, 64, spare=5)
    q, kn, vn = (x.cuda() for x in round_inputs(g, 2, 5, 4, 2, 64, "bf16"))
    logits = torch.randn(2, 3, 400, generator=g).cuda()
    tokens = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    calls = dict(attention=lambda **kw: sv.verify_attention(q, p.cache, p.dtable, p.dlens, k=kn, v=vn, lse=True, **kw),
                 logits=lambda **kw: sv.process_logits(logits, tokens=tokens, **kw),
                 write=lambda **kw: sv.kv_cache_write(kn, vn, p.cache, p.dtable, p.dlens, **kw),
                 read=lambda **kw: sv.kv_cache_read(p.cache, p.dtable, p.dlens, max_len=90, dtype=torch.float32, **kw))
    call = calls[what]
    want = call()
    st = torch.cuda.Stream()
    call(stream=st)  # its workspace is there from now on
    for name, t in want.items():
        busy_block(t.numel() * t.element_size(), 77)
        got = call(stream=st)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]), (name, n)


def test_a_new_workspace_on_another_stream_is_the_calls_own():
    g = torch.Generator().manual_seed(72)
    p = Pool(g, [3000, 130], 2, 32, 64)
    q, kn, vn = (x.cuda() for x in round_inputs(g, 2, 5, 4, 2, 64, "bf16"))
    call = lambda **kw: sv.verify_attention(q, p.cache, p.dtable, p.dlens, k=kn, v=vn, lse=True, **kw)
    out = {n: torch.empty_like(t) for n, t in call().items()}
    n = B_.load().verify_attention_workspace_bytes(2, 5, 4, 2, 64)
    old = dict(B_._round_ws)
    B_._round_ws.clear()
    try:
        st = torch.cuda.Stream()
        at = busy_block(n, 77)
        call(stream=st, out=out)
        (buf,) = B_._round_ws.values()
        assert buf.data_ptr() + buf.numel() <= at or at + n <= buf.data_ptr()
        torch.cuda.synchronize()
    finally:
        B_._round_ws.update(old)


class Spy:
    """The library, noting the workspace of every verify_attention."""

    def __init__(self, lib):
        self.lib, self.seen = lib, []

    def __getattr__(self, name):
        f = getattr(self.lib, name)
        if name != "verify_attention":
            return f

        def call(*a):
            self.seen.append((a[-3], a[-2]))
            return f(*a)
        return call


@pytest.mark.parametrize("T,hq,other", [(3, 8, False), (6, 16, False), (6, 16, True)])
def test_captured_attention_has_a_workspace_of_its_own(monkeypatch, T, hq, other):
    """Two graphs captured without a workspace, replayed at the same time on two streams while eager calls run."""
    g = torch.Generator().manual_seed(73)
    spy = Spy(B_.load())
    monkeypatch.setattr(B_, "load", lambda *a: spy)
    cases, graphs = [], []
    for seed in range(2):
        p = Pool(g, [5000 + 900 * seed, 100], 2, 64, 128)
        q, kn, vn = (x.cuda() for x in round_inputs(g, 2, T, hq, 2, 128, "bf16"))
        cases.append(lambda p=p, q=q, kn=kn, vn=vn, **kw: sv.verify_attention(q, p.cache, p.dtable, p.dlens, k=kn, v=vn, lse=True, **kw))
    want = [c() for c in cases]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if other:  # a branch of the capture
                side.wait_stream(torch.cuda.current_stream())
                r = c(stream=side)
                torch.cuda.current_stream().wait_stream(side)
            else:
                r = c()
        graphs.append((graph, r))
    eager, a, b = ((x, x + n) for x, n in spy.seen[1:4])
    for x, y in ((eager, a), (eager, b), (a, b)):
        assert x[1] <= y[0] or y[1] <= x[0], spy.seen
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for st, (graph, r) in zip(streams, graphs):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                for t in r.values():
                    t.zero_()
                graph.replay()
        now = [c() for c in cases]
        torch.cuda.synchronize()
        for w, (_, r), e in zip(want, graphs, now):
            for n in w:
                assert torch.equal(r[n], w[n]) and torch.equal(e[n], w[n]), n


def test_a_larger_workspace_leaves_captured_calls_alone():
    """64 channels captured, then 128 channels eagerly on the same stream, whose workspace is larger."""
    g = torch.Generator().manual_seed(74)
    st = torch.cuda.Stream()
    calls = []
    for D in (64, 128):
        p = Pool(g, [4000, 100], 2, 64, D)
        q, kn, vn = (x.cuda() for x in round_inputs(g, 2, 6, 16, 2, D, "bf16"))
        calls.append(lambda p=p, q=q, kn=kn, vn=vn, **kw: sv.verify_attention(q, p.cache, p.dtable, p.dlens, k=kn, v=vn, lse=True, **kw))
    want = calls[0]()
    old = dict(B_._round_ws)
    B_._round_ws.clear()
    try:
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            calls[0]()
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=st):
                r = calls[0]()
            calls[1]()
            torch.cuda.synchronize()
            n = B_.load().verify_attention_workspace_bytes(2, 6, 16, 2, 64)
            held = torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")  # takes what the smaller one left
            graph.replay()
            torch.cuda.synchronize()
            assert bool((held == 0x7f).all())
        for n in want:
            assert torch.equal(r[n], want[n]), n
    finally:
        B_._round_ws.update(old)


# ------------------------------------------------------------------ logits

@pytest.mark.parametrize("rep", [1.3, 0.7, 1.1754944e-38, 1e-40, 2.9387359e-39, 3e38])
def test_logits_are_divided_by_the_repetition_penalty(rep):
    """The quotient rounded once, also where the reciprocal is no normal number."""
    g = torch.Generator().manual_seed(81)
    V = 4099
    x = torch.randn(1, 2, V, generator=g) * torch.exp2(torch.randint(-60, 4, (V,), generator=g).float())
    hist = torch.randperm(V, generator=g).to(torch.int32)[None, :4000].contiguous()
    r = torch.tensor([rep])
    y = sv.process_logits(x.cuda(), tokens=torch.zeros(1, 1, dtype=torch.int32, device="cuda"), history=hist.cuda(),
                          repetition=r.cuda())["logits"].cpu()
    hit = torch.zeros(V, dtype=torch.bool)
    hit[hist[0].long()] = True
    for row in range(2):
        seen = hit.clone()
        if row:
            seen[0] = True
        want = torch.where(seen, torch.where(x[0, row] > 0, x[0, row] / r, x[0, row] * r), x[0, row])
        assert torch.equal(y[0, row], want)
