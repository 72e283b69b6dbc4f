"""The operators around one verification round: what is timed, on which sizes, in plain form and as the library's calls.

Four operators make up the target's side of a speculative round next to the verify calls:

  attn    verify_attention   attention of the round's rows over the 8-bit paged cache and the round's own rows
  logits  process_logits     penalties, biases and grammar masks on the rows the verify calls read
  write   kv_cache_write     quantises the accepted rows into the cache
  read    kv_cache_read      reads a cache back

The cache holds e4m3 codes in pages [P, Hkv, page, D] and one fp32 scale, a power of two, per page and head.
"""
import math
import random

import torch

own = False  # set by the tools: False computes the plain form, True makes the library's calls

FP8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E_MIN, E_MAX = -60, 60  # a page's scale is 2^e with e in this range


def listed():
    return [
        # one request decoding without a draft, after a short prompt: latency alone
        dict(name="attn_token", op="attn", B=1, T=1, hq=32, hkv=8, D=128, page=64, L=1023, tree=False, dtype="bf16"),
        # a batch whose requests verify five drafted tokens each, ragged contexts
        dict(name="attn_draft", op="attn", B=32, T=6, hq=32, hkv=8, D=128, page=64, L=8192, tree=False, dtype="bf16"),
        # the same round with eight query heads a cache head, small pages and an odd context
        dict(name="attn_draft_g8", op="attn", B=64, T=6, hq=64, hkv=8, D=128, page=16, L=4099, tree=False, dtype="bf16"),
        # the tree workload: 64 candidate nodes and the frontier row a request
        dict(name="attn_tree", op="attn", B=32, T=65, hq=32, hkv=8, D=128, page=64, L=4096, tree=True, dtype="bf16"),
        # one long document, few rows: the work has to be split over the context
        dict(name="attn_long", op="attn", B=1, T=5, hq=16, hkv=2, D=64, page=32, L=131071, tree=False, dtype="f16"),
        # one request, next token, small vocabulary: latency alone
        dict(name="logits_token", op="logits", B=1, R=1, V=32000, H=600, nb=8, mask=False, tree=False, dtype="bf16"),
        # the target rows of a drafted round at the large vocabulary
        dict(name="logits_draft", op="logits", B=64, R=6, V=128256, H=2048, nb=64, mask=False, tree=False, dtype="bf16"),
        # the rows of a candidate tree under a grammar
        dict(name="logits_tree", op="logits", B=32, R=65, V=128256, H=4000, nb=0, mask=True, tree=True, dtype="bf16"),
        # the commit after a drafted round: one to six accepted rows a request, into pages partly filled
        dict(name="write_round", op="write", B=64, T=6, hkv=8, D=128, page=64, L=3000, nodes=True, dtype="bf16"),
        # prompts of several thousand tokens
        dict(name="write_prompt", op="write", B=4, T=8191, hkv=8, D=128, page=64, L=0, nodes=False, dtype="bf16"),
        # a short prefix handed to another program
        dict(name="read_prefix", op="read", B=2, L=333, hkv=4, D=64, page=16, dtype="f16"),
        # a batch's whole cache, for a pass that wants 16-bit keys and values
        dict(name="read_batch", op="read", B=16, L=12289, hkv=8, D=128, page=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "logits", "write", "read"])
    if op == "attn":
        while True:
            hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
            c = dict(op=op, B=_log(rng, 1, 64), T=rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 2, 65)]), hq=hkv * group, hkv=hkv,
                     D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), L=_log(rng, 1, 131072), tree=rng.random() < 0.4,
                     dtype=rng.choice(["bf16", "bf16", "f16"]))
            if c["B"] * c["L"] * hkv * c["D"] <= 3e8 and c["B"] * c["L"] * c["hq"] * c["D"] * c["T"] <= 3e10:
                return c
    if op == "logits":
        while True:
            R = rng.choice([1, _log(rng, 2, 9), _log(rng, 2, 65)])
            c = dict(op=op, B=_log(rng, 1, 64), R=R, V=_log(rng, 1000, 160000), H=_log(rng, 1, 8192), nb=rng.choice([0, 1, 37, 300]),
                     mask=rng.random() < 0.5, tree=R > 1 and rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]))
            if c["B"] * R * c["V"] * (2 if c["dtype"] == "f32" else 1) <= 2.4e8:
                return c
    if op == "write":
        long = rng.random() < 0.4
        while True:
            c = dict(op=op, B=_log(rng, 1, 128), T=_log(rng, 100, 8192) if long else _log(rng, 1, 65), hkv=rng.choice([1, 2, 4, 8]),
                     D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), L=rng.choice([0, _log(rng, 1, 4096)]),
                     nodes=not long and rng.random() < 0.5, dtype=rng.choice(["bf16", "f16", "f32"]))
            if c["B"] * c["T"] * c["hkv"] * c["D"] * (2 if c["dtype"] == "f32" else 1) <= 3.3e7 and c["B"] * (c["L"] + c["T"]) * c["hkv"] * c["D"] <= 2.7e8:
                return c
    while True:
        c = dict(op=op, B=_log(rng, 1, 64), L=_log(rng, 1, 16384), hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]),
                 page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "f16", "f32"]))
        if c["B"] * c["L"] * c["hkv"] * c["D"] * (2 if c["dtype"] == "f32" else 1) <= 2e8:
            return c


# ---- sizes that follow from the case alone (ragged lengths, accepted rows)

def _lens(c):
    """Context lengths: the longest is L, the others spread between a quarter of it and all of it."""
    return [c["L"] if b == 0 else max(min(c["L"], 1), int(c["L"] * (0.25 + 0.75 * ((b * 0.6180339887) % 1.0)))) for b in range(c["B"])]


def _hist_lens(c):
    return [max(1, int(c["H"] * (0.3 + 0.7 * ((b * 0.7548776662) % 1.0)))) for b in range(c["B"])]


def _accepted(c):
    """Accepted drafts a request: all of the prompt's rows, or 0 .. T-1 of a round's."""
    if c["T"] > 65:
        return [c["T"] - 1 - (b * 37) % max(1, c["T"] // 4) for b in range(c["B"])]
    return [(b * 5 + 2) % c["T"] for b in range(c["B"])]


def work(case):
    c = case
    e = {"bf16": 2, "f16": 2, "f32": 4}[c["dtype"]]
    if c["op"] == "attn":
        L = sum(_lens(c))
        pages = sum(-(-n // c["page"]) for n in _lens(c))
        rows = c["B"] * c["T"]
        by = 2 * L * c["hkv"] * c["D"] + 8 * pages * c["hkv"] + 4 * pages + rows * c["D"] * e * (2 * c["hq"] + 2 * c["hkv"]) + 4 * rows * c["hq"]
        seen = c["T"] * L + (c["B"] * c["T"] * (c["T"] + 1) // 2 if not c["tree"] else rows * 4)
        return {"bytes": by, "flops": 4 * c["hq"] * c["D"] * seen}
    if c["op"] == "logits":
        n = c["B"] * c["R"] * c["V"]
        by = 2 * n * e + (c["B"] * c["R"] * (-(-c["V"] // 32)) * 4 if c["mask"] else 0) + 4 * sum(_hist_lens(c)) + 8 * c["B"] * c["nb"]
        return {"bytes": by, "flops": 4 * n}
    if c["op"] == "write":
        n = 2 * sum(a + 1 for a in _accepted(c)) * c["hkv"] * c["D"]
        return {"bytes": n * (e + 1), "flops": 3 * n}
    n = 2 * sum(_lens(c)) * c["hkv"] * c["D"]
    full = 2 * c["B"] * c["L"] * c["hkv"] * c["D"]
    return {"bytes": n + full * e, "flops": n}


# ---- inputs

def _kv(g, shape, dtype):
    """Keys or values as a model makes them: unit normal, some channels far larger than the rest, some tokens too."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    ch = torch.exp(0.5 * torch.randn(shape[-1:], generator=g, device="cuda"))
    tok = torch.exp(0.3 * torch.randn(shape[:2] + (1,) * (len(shape) - 2), generator=g, device="cuda"))
    return (x * ch * tok).to(dtype)


def _scale_exp(amax):
    """The smallest e with amax <= 448 * 2^e, in [E_MIN, E_MAX]."""
    m, x = torch.frexp(amax)  # amax = m * 2^x, m in [0.5, 1)
    e = torch.where(m > 0.875, x - 8, x - 9)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _filled_cache(g, c, lens, spare):
    """A cache whose requests hold `lens` tokens, in pages scattered over the pool, and its page table."""
    per = [-(-(n + spare) // c["page"]) for n in lens]
    P, width = sum(per) + 3, max(1, max(per))
    perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(c["B"], width, dtype=torch.int64)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    table = perm[table.cuda()]
    out = {"table": table.contiguous(), "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    for n in ("k", "v"):
        codes = torch.empty(P, c["hkv"], c["page"], c["D"], dtype=FP8, device="cuda")
        scales = torch.empty(P, c["hkv"], device="cuda")
        step = max(1, (1 << 27) // (c["hkv"] * c["page"] * c["D"]))
        for p in range(0, P, step):
            x = _kv(g, (min(step, P - p), c["hkv"], c["page"], c["D"]), torch.float32)
            e = _scale_exp(x.abs().amax((2, 3)))
            codes[p:p + step] = torch.ldexp(x, -e[:, :, None, None]).to(FP8)
            scales[p:p + step] = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
        out[n], out[n + "_scale"] = codes, scales
    return out


def _parents(g, B, N):
    """Ancestor-closed candidate trees: a node's parent is the frontier (-1) or any earlier node."""
    at = torch.arange(N, device="cuda")
    u = torch.rand(B, N, generator=g, device="cuda")
    return ((u * (at + 1)).long().clamp(max=N - 1).minimum(at) - 1).to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    dt = DTYPES[c["dtype"]]
    if c["op"] == "attn":
        s.update(_filled_cache(g, c, _lens(c), 0))
        B, T = c["B"], c["T"]
        s["q"] = (1.5 * torch.randn(B, T, c["hq"], c["D"], generator=g, device="cuda")).to(dt)
        s["kn"], s["vn"] = _kv(g, (B, T, c["hkv"], c["D"]), dt), _kv(g, (B, T, c["hkv"], c["D"]), dt)
        s["parents"] = _parents(g, B, T - 1) if c["tree"] else None
    elif c["op"] == "logits":
        B, R, V = c["B"], c["R"], c["V"]
        s["logits"] = torch.empty(B, R, V, dtype=dt, device="cuda")
        for b in range(B):
            s["logits"][b] = (3 * torch.randn(R, V, generator=g, device="cuda")).to(dt)
        # a text repeats its own words: tokens of a skewed law
        words = torch.rand(B, c["H"] + R, generator=g, device="cuda").pow(3).mul(min(V, 5000)).long()
        words = words * (V // min(V, 5000))
        s["history"], s["tokens"] = words[:, :c["H"]].to(torch.int32).contiguous(), words[:, c["H"]:c["H"] + R - 1].to(torch.int32).contiguous()
        s["hist_len"] = torch.tensor(_hist_lens(c), dtype=torch.int32, device="cuda")
        s["prompt_len"] = (s["hist_len"] // 3).to(torch.int32)
        s["parents"] = _parents(g, B, R - 1) if c["tree"] else None
        s["rep"] = 1 + 0.3 * torch.rand(B, generator=g, device="cuda")
        s["pres"], s["freq"] = (0.8 * torch.rand(B, generator=g, device="cuda") for _ in range(2))
        s["bias_tokens"] = s["bias_values"] = s["allowed"] = None
        if c["nb"]:
            s["bias_tokens"] = torch.stack([torch.randperm(V, generator=g, device="cuda")[:c["nb"]] for _ in range(B)]).to(torch.int32)
            s["bias_values"] = 5 * torch.randn(B, c["nb"], generator=g, device="cuda")
        if c["mask"]:
            s["allowed"] = torch.randint(-2**31, 2**31, (B, R, -(-V // 32)), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    elif c["op"] == "write":
        s.update(_filled_cache(g, c, _lens(c), c["T"]))
        B, T = c["B"], c["T"]
        s["kn"], s["vn"] = _kv(g, (B, T, c["hkv"], c["D"]), dt), _kv(g, (B, T, c["hkv"], c["D"]), dt)
        s["accepted"] = torch.tensor(_accepted(c), dtype=torch.int32, device="cuda")
        s["nodes"] = None
        if c["nodes"]:  # an accepted path: ascending node ids, then -1
            ids = torch.rand(B, T - 1, generator=g, device="cuda").argsort(1)
            keep = torch.arange(T - 1, device="cuda")[None] < s["accepted"][:, None]
            ids = torch.where(keep, ids, torch.full_like(ids, T)).sort(1).values
            s["nodes"] = torch.where(keep, ids, torch.full_like(ids, -1)).to(torch.int32)
    else:
        s.update(_filled_cache(g, c, _lens(c), 0))
    return s


# ---- one pass

def _lib():
    import speculative_decoding_verification_spec_gb300 as sv

    return sv


def _cache(s):
    return s["k"], s["v"], s["k_scale"], s["v_scale"]


def run(s):
    return {"attn": _attn, "logits": _logits, "write": _write, "read": _read}[s["case"]["op"]](s)


def _sees(s, T):
    """[B or 1, T, T]: whether row t of the round sees row j of it."""
    at = torch.arange(T, device="cuda")
    if s["parents"] is None:
        return (at[None, :] <= at[:, None])[None]
    B = s["parents"].shape[0]
    up = torch.zeros(B, T, T, device="cuda")
    up[:, 1:].scatter_(2, (s["parents"].long() + 1)[:, :, None], 1.0)  # row t's predecessor
    reach = up + torch.eye(T, device="cuda")
    for _ in range(max(1, (T - 1).bit_length())):
        reach = (reach @ reach).clamp(max=1.0)
    return reach > 0


def _gathered(s, n):
    """The cache's values along each request, [B, Hkv, tokens, D] in 32 bits."""
    c = s["case"]
    t = s["table"].long()
    x = s[n].view(torch.uint8)[t].view(FP8).float() * s[n + "_scale"][t][..., None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(c["B"], c["hkv"], -1, c["D"])


def _attn(s):
    c = s["case"]
    scale = 1.0 / math.sqrt(c["D"])
    if own:
        r = _lib().verify_attention(s["q"], _cache(s), s["table"], s["lens"], k=s["kn"], v=s["vn"], parents=s["parents"], scale=scale, lse=True)
        return {"out": r["out"], "lse": r["lse"]}
    B, T, G = c["B"], c["T"], c["hq"] // c["hkv"]
    q = s["q"].float().view(B, T, c["hkv"], G, c["D"]).permute(0, 2, 1, 3, 4).reshape(B, c["hkv"], T * G, c["D"])
    k = torch.cat([_gathered(s, "k"), s["kn"].float().transpose(1, 2)], 2)
    v = torch.cat([_gathered(s, "v"), s["vn"].float().transpose(1, 2)], 2)
    old = (torch.arange(k.shape[2] - T, device="cuda")[None] < s["lens"][:, None])[:, None].expand(B, T, -1)
    mask = torch.cat([old, _sees(s, T).expand(B, T, T)], 2)[:, None, :, None].expand(B, 1, T, G, -1).reshape(B, 1, T * G, -1)
    p = (q @ k.transpose(2, 3) * scale).masked_fill_(~mask, float("-inf"))
    m = p.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(p.sub_(m))
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / l
    lse = (m + torch.log(l))[..., 0]
    back = lambda x: x.view(B, c["hkv"], T, G, -1).permute(0, 2, 1, 3, 4).reshape(B, T, c["hq"], -1)
    return {"out": back(o).to(s["q"].dtype), "lse": back(lse)[..., 0].contiguous()}


def _logits(s):
    c = s["case"]
    if own:
        r = _lib().process_logits(s["logits"], tokens=s["tokens"], parents=s["parents"], history=s["history"], prompt_len=s["prompt_len"],
                                   history_len=s["hist_len"], repetition=s["rep"], presence=s["pres"], frequency=s["freq"],
                                   bias_tokens=s["bias_tokens"], bias_values=s["bias_values"], allowed=s["allowed"])
        return r["logits"]
    B, R, V = c["B"], c["R"], c["V"]
    at = torch.arange(c["H"], device="cuda")[None]
    live = at < s["hist_len"][:, None]
    outp = (live & (at >= s["prompt_len"][:, None])).float()
    hist = s["history"].long()
    base = torch.zeros(B, V, device="cuda").scatter_add_(1, hist, outp)
    said = torch.zeros(B, V, device="cuda").scatter_add_(1, hist, live.float())
    count = base[:, None].repeat(1, R, 1)
    if R > 1:
        count.scatter_add_(2, s["tokens"].long()[:, None].expand(B, R, R - 1), _sees(s, R)[:, :, 1:].float().expand(B, R, R - 1))
    x = s["logits"].float()
    rep = s["rep"][:, None, None]
    x = torch.where((count > 0) | (said[:, None] > 0), torch.where(x > 0, x / rep, x * rep), x)
    x = x - (s["freq"][:, None, None] * count + s["pres"][:, None, None] * (count > 0))
    if c["nb"]:
        x = x + torch.zeros(B, V, device="cuda").scatter_(1, s["bias_tokens"].long(), s["bias_values"])[:, None]
    if c["mask"]:
        bit = (s["allowed"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        x = x.masked_fill(bit.view(B, R, -1)[..., :V] == 0, float("-inf"))
    return x.to(s["logits"].dtype)


def _write(s):
    c = s["case"]
    if own:
        r = _lib().kv_cache_write(s["kn"], s["vn"], _cache(s), s["table"], s["lens"], accepted_len=s["accepted"], out_nodes=s["nodes"])
        return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "lens": r["lens"]}
    B, T, pg = c["B"], c["T"], c["page"]
    n = s["accepted"].long() + 1
    i = torch.arange(T, device="cuda")[None].expand(B, T)
    row = i if s["nodes"] is None else torch.cat([i[:, :1] * 0, s["nodes"].long() + 1], 1)
    live = i < n[:, None]
    pos = s["lens"].long()[:, None] + i
    j = (pos // pg).clamp(max=s["table"].shape[1] - 1)
    page, slot = s["table"].long().gather(1, j), pos % pg
    b_of = torch.arange(B, device="cuda")[:, None].expand(B, T)
    page, slot, row, b_of, pos = page[live], slot[live], row[live], b_of[live], pos[live]
    for name, x in (("k", s["kn"]), ("v", s["vn"])):
        codes, scales = s[name], s[name + "_scale"]
        new = x[b_of, row].float()  # [rows, Hkv, D]
        big = new.abs()
        amax = torch.where(big <= 448.0 * 2.0**E_MAX, big, torch.zeros_like(big)).amax(2)
        top = torch.zeros_like(scales).scatter_reduce_(0, page[:, None].expand(-1, c["hkv"]), amax, "amax")
        touched = torch.zeros(len(scales), dtype=torch.bool, device="cuda").index_fill_(0, page, True)
        # tokens that a page held before: the request's length ends inside it
        held = torch.zeros(len(scales), dtype=torch.int64, device="cuda")
        held.scatter_reduce_(0, page, (slot - (pos - s["lens"].long()[b_of])).clamp(min=0), "amax")
        e = _scale_exp(top)
        fresh = torch.ldexp(torch.ones_like(scales), e)
        fresh = torch.where((held > 0)[:, None], torch.maximum(fresh, scales), fresh)
        fresh = torch.where(touched[:, None], fresh, scales)
        grown = torch.nonzero(touched & (held > 0))[:, 0]
        raw = codes.view(torch.uint8)
        was = raw[grown].view(FP8).float()
        keep = (torch.arange(pg, device="cuda")[None] < held[grown][:, None])[:, None, :, None]
        raw[grown] = torch.where(keep, was * (scales / fresh)[grown][..., None, None], was).to(FP8).view(torch.uint8)
        scales.copy_(fresh)
        y = new / fresh[page][..., None]
        raw[page, :, slot] = torch.where(y.abs() <= 448.0, y, torch.full_like(y, float("nan"))).to(FP8).view(torch.uint8)
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "lens": (s["lens"].long() + n).to(torch.int32)}


def _read(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if own:
        r = _lib().kv_cache_read(_cache(s), s["table"], s["lens"], max_len=c["L"], dtype=dt)
        return {"k": r["k"], "v": r["v"]}
    live = (torch.arange(c["L"], device="cuda")[None] < s["lens"][:, None])[:, :, None, None]
    return {n: _gathered(s, n)[:, :, :c["L"]].transpose(1, 2).masked_fill(~live, 0.0).to(dt).contiguous() for n in ("k", "v")}


# ---- the definitions in 64 bits, one request (and head) at a time

def _line(s, n, b, length):
    pg = s["case"]["page"]
    ids = s["table"][b, :-(-length // pg)].long()
    x = s[n].view(torch.uint8)[ids].view(FP8).double() * s[n + "_scale"][ids].double()[:, :, None, None]  # [pages, Hkv, page, D]
    return x.transpose(0, 1).flatten(1, 2)[:, :length]


def _path_rows(parents, b, t):
    """Row t and the rows before it on its path, the frontier row 0 last."""
    rows = [t]
    while rows[-1] > 0:
        rows.append(rows[-1] - 1 if parents is None else parents[b][rows[-1] - 1] + 1)
    return rows


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    par = None
    if s.get("parents") is not None:
        par = s["parents"].tolist()
    if c["op"] == "attn":
        B, T, G = c["B"], c["T"], c["hq"] // c["hkv"]
        out = torch.zeros(B, T, c["hq"], c["D"], dtype=torch.float64, device="cuda")
        lse = torch.zeros(B, T, c["hq"], dtype=torch.float64, device="cuda")
        lens = _lens(c)
        for b in range(B):
            k, v = _line(s, "k", b, lens[b]), _line(s, "v", b, lens[b])
            see = torch.zeros(T, T, dtype=torch.bool)
            for t in range(T):
                see[t, _path_rows(par, b, t)] = True
            bar = torch.where(see, 0.0, -math.inf).double().cuda()
            for h in range(c["hkv"]):
                kk, vv = torch.cat([k[h], s["kn"][b, :, h].double()]), torch.cat([v[h], s["vn"][b, :, h].double()])
                for x in range(h * G, h * G + G):
                    z = torch.matmul(s["q"][b, :, x].double(), kk.T) / math.sqrt(c["D"])
                    z[:, lens[b]:] += bar
                    lse[b, :, x] = torch.logsumexp(z, 1)
                    out[b, :, x] = torch.matmul(torch.exp(z - lse[b, :, x, None]), vv)
        return {"out": out, "lse": lse}
    if c["op"] == "logits":
        if c["B"] * c["R"] > 600:
            return None
        y = s["logits"].double()
        ar = torch.arange(c["V"], device="cuda")
        hist, toks, hl, pl = s["history"].tolist(), s["tokens"].tolist(), s["hist_len"].tolist(), s["prompt_len"].tolist()
        for b in range(c["B"]):
            base = torch.bincount(torch.tensor(hist[b][pl[b]:hl[b]], dtype=torch.int64), minlength=c["V"])
            known = torch.bincount(torch.tensor(hist[b][:hl[b]], dtype=torch.int64), minlength=c["V"]) > 0
            base, known = base.cuda(), known.cuda()
            rep, fr, pr = (float(s[n][b]) for n in ("rep", "freq", "pres"))
            for r in range(c["R"]):
                path = torch.tensor([toks[b][w - 1] for w in _path_rows(par, b, r) if w > 0], dtype=torch.int64)
                n = base + torch.bincount(path, minlength=c["V"]).cuda()
                z = y[b, r]
                hit = known | (n > 0)
                z[hit] = torch.where(z[hit] > 0, z[hit] / rep, z[hit] * rep)
                z -= fr * n + pr * (n > 0)
                if c["nb"]:
                    z[s["bias_tokens"][b].long()] += s["bias_values"][b].double()
                if c["mask"]:
                    z[(s["allowed"][b, r][ar // 32] >> (ar % 32).int()) & 1 == 0] = -math.inf
        return y
    if c["op"] == "write":
        if c["B"] * c["T"] > 40000:
            return None
        res = {"lens": None}
        lens, acc = _lens(c), _accepted(c)
        table = s["table"].tolist()
        nodes = s["nodes"].tolist() if s["nodes"] is not None else None
        for name, x in (("k", s["kn"]), ("v", s["vn"])):
            codes, scales = s[name].double(), s[name + "_scale"].double()
            for b in range(c["B"]):
                rows = [0] + [nodes[b][i] + 1 if nodes else i + 1 for i in range(acc[b])]
                at = 0
                while at < len(rows):
                    j, first = divmod(lens[b] + at, c["page"])
                    take = rows[at:at + c["page"] - first]
                    at += len(take)
                    new = x[b, take].double().transpose(0, 1)  # [Hkv, rows, D]
                    m, e = torch.frexp(new.abs().amax((1, 2)) / 448.0)
                    e = torch.where(m == 0.5, e - 1, e).clamp(E_MIN, E_MAX)  # ceil(log2), exact at powers of two
                    sc, p = torch.ldexp(torch.ones_like(m), e), table[b][j]
                    if first:
                        sc = torch.maximum(sc, scales[p])
                        codes[p, :, :first] *= (scales[p] / sc)[:, None, None]
                    scales[p] = sc
                    codes[p, :, first:first + len(take)] = new / sc[:, None, None]
            res[name], res[name + "_scale"] = codes, scales
        return res
    out = {n: torch.zeros(c["B"], c["L"], c["hkv"], c["D"], dtype=torch.float64, device="cuda") for n in ("k", "v")}
    for b, length in enumerate(_lens(c)):
        for n in ("k", "v"):
            out[n][b, :length] = _line(s, n, b, length).transpose(0, 1)
    return out
