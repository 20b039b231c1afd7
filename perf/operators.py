"""Cases of the 4-bit KV cache and cache-eviction operators, their plain forms
and the calls a user makes of them.

Four operators over the paged cache [num_blocks, Hkv, 16, row]:

  append  kv_append of new K/V rows into a cache, and kv_gather of the rows
          just written (what the cache now holds, as values)
  attend  paged_decode_attention / paged_tree_attention over a 4-bit cache
  score   paged_score_update: the attention weight every cached key received
          from the new query rows, added to its running score
  evict   kv_evict: each (sequence, kv head) keeps its sinks, its newest rows
          and the best-scored rest, compacted into destination pages

A 4-bit row of D elements is D/2 bytes of E2M1 codes (element 2i in the low
nibble of byte i) followed by D/16 E4M3 scales, one per 16 elements:
value = code * scale * k_scale (v_scale).  A new row x is stored as
y = x / k_scale (fp32), scale = E4M3(max|y| / 6) of its 16 elements kept in
[2^-9, 448], code = E2M1(y / scale), every quotient in fp32 and every
rounding to nearest, ties to even, saturating.
"""
import math

import torch

own = False

PAGE = 16
GROUP = 16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
FP8_SCALE = 2.0 ** -5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step's new rows of the 32-sequence, 32-head decode shape:
        # a few hundred KB, the latency of two short launches
        dict(name="append step", op="append", dtype="fp4", batch=32, hkv=32,
             d=128, n_new=1, ctx_min=512, ctx_max=4096, k_scale=1.0),
        # prompt chunks of 64 rows entering the cache, GQA heads
        dict(name="append chunk", op="append", dtype="fp4", batch=64, hkv=8,
             d=128, n_new=64, ctx_min=64, ctx_max=2048, k_scale=0.0371),
        # the smallest attention call: one short sequence, head_dim 64
        dict(name="attend tiny", op="attend", batch=1, hq=4, hkv=4, d=64,
             q_len=1, ctx_min=250, ctx_max=250, n_sink=0, window=0,
             tree=False, k_scale=1.0),
        # ordinary decode, one query row per kv head, ragged contexts
        dict(name="attend decode", op="attend", batch=32, hq=32, hkv=32,
             d=128, q_len=1, ctx_min=512, ctx_max=4096, n_sink=0, window=0,
             tree=False, k_scale=1.0),
        # verification of 4 drafts and the bonus position, GQA group 4
        dict(name="attend verify", op="attend", batch=16, hq=32, hkv=8,
             d=128, q_len=5, ctx_min=2048, ctx_max=8192, n_sink=0, window=0,
             tree=False, k_scale=0.0371),
        # a draft tree of 15 nodes: 60 query rows per kv head
        dict(name="attend tree", op="attend", batch=16, hq=32, hkv=8, d=128,
             q_len=15, ctx_min=2048, ctx_max=8192, n_sink=0, window=0,
             tree=True, k_scale=1.0),
        # long contexts, few sequences: each group split over many SMs
        dict(name="attend long", op="attend", batch=4, hq=64, hkv=8, d=128,
             q_len=1, ctx_min=131072, ctx_max=131072, n_sink=0, window=0,
             tree=False, k_scale=1.0),
        # weights of a decode step over a bf16 cache
        dict(name="score decode", op="score", dtype="bf16", batch=32, hq=32,
             hkv=32, d=128, q_len=1, ctx_min=512, ctx_max=4096, n_sink=0,
             window=0, tree=False, k_scale=1.0),
        # weights of a verification step over a 4-bit cache
        dict(name="score verify", op="score", dtype="fp4", batch=16, hq=32,
             hkv=8, d=128, q_len=5, ctx_min=2048, ctx_max=8192, n_sink=0,
             window=0, tree=False, k_scale=1.0),
        # one sequence a little over its budget
        dict(name="evict small", op="evict", dtype="bf16", batch=1, hkv=8,
             d=128, ctx_min=1087, ctx_max=1087, budget=1024, n_sink=4,
             n_recent=128),
        # the decode shape cut to half of its longest context
        dict(name="evict decode", op="evict", dtype="bf16", batch=32, hkv=32,
             d=128, ctx_min=2200, ctx_max=4096, budget=2048, n_sink=4,
             n_recent=512),
        # long 4-bit contexts cut to an eighth
        dict(name="evict long", op="evict", dtype="fp4", batch=4, hkv=8,
             d=128, ctx_min=120000, ctx_max=131072, budget=16384, n_sink=4,
             n_recent=4096),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = max(work(c)["bytes"] for c in listed())
    flops = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(("append", "attend", "attend", "score", "evict"))
        hkv = rng.choice((1, 2, 3, 4, 8, 8, 16, 32))
        group = rng.choice((1, 1, 2, 3, 4, 4, 5, 7, 8))
        d = rng.choice((64, 128, 128))
        batch = _log_int(rng, 1, 48)
        hi = _log_int(rng, 40, 131072)
        lo = max(17, int(hi * rng.uniform(0.2, 1.0)))
        k_scale = rng.choice((1.0, 1.0, 0.0371, 0.4))
        c = dict(op=op, batch=batch, hkv=hkv, d=d, ctx_min=lo, ctx_max=hi)
        if op == "append":
            c.update(dtype=rng.choice(("fp4", "fp4", "fp4", "bf16", "fp8", "f32")),
                     n_new=rng.randint(1, 64), k_scale=k_scale)
            c["ctx_max"] = min(hi, 8192)
            c["ctx_min"] = max(c["n_new"], min(lo, c["ctx_max"]))
            c["ctx_max"] = max(c["ctx_min"], c["ctx_max"])
        elif op == "evict":
            c.update(dtype=rng.choice(("fp4", "bf16", "fp8", "f32")))
            c["budget"] = max(2, int(hi * rng.uniform(0.1, 1.0)))
            c["n_sink"] = rng.randint(0, min(8, c["budget"] // 2))
            c["n_recent"] = int((c["budget"] - c["n_sink"]) * rng.uniform(0.0, 0.6))
        else:
            tree = rng.random() < 0.25
            c.update(hq=hkv * group, q_len=rng.choice((1, 1, 2, 3, 5, 8, 11, 16)),
                     tree=tree, n_sink=0, window=0, k_scale=k_scale)
            if not tree and rng.random() < 0.3:
                c.update(n_sink=rng.randint(0, 20),
                         window=rng.randint(1, max(1, hi)))
            if op == "score":
                c["dtype"] = rng.choice(("fp4", "bf16", "fp8", "f32"))
                if c["dtype"] != "fp4":
                    c["k_scale"] = FP8_SCALE if c["dtype"] == "fp8" else 1.0
        w = work(c)
        # cached elements bound the plain form's memory
        cells = batch * c["ctx_max"] * hkv * d
        if (w["bytes"] <= top and w["flops"] <= flops and cells <= 600e6 and
                cells * c.get("hq", hkv) / hkv * c.get("q_len", 1) <= 16e9):
            return c


# --------------------------------------------- the 4-bit format, elementary

def _quantise(y):
    """fp32 y [..., D] -> (codes uint8 [..., D], scales e4m3 [..., D/16])."""
    blocks = y.unflatten(-1, (-1, GROUP))
    amax = blocks.abs().amax(-1)
    scale = (amax / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    scale = scale.clamp(min=2.0 ** -9)
    r = blocks.abs() / scale[..., None]
    code = ((r > 0.25).to(torch.uint8) + (r >= 0.75) + (r > 1.25) + (r >= 1.75) +
            (r > 2.5) + (r >= 3.5) + (r > 5.0))
    code = code | (blocks < 0).to(torch.uint8) * 8
    return code.flatten(-2), scale.to(torch.float8_e4m3fn)


def _pack(code, scale):
    byte = code[..., 0::2] | (code[..., 1::2] << 4)
    return torch.cat((byte, scale.view(torch.uint8)), -1)


def _unpack(row, d):
    """Rows [..., D/2 + D/16] uint8 -> code * scale, fp32 [..., D]."""
    byte = row[..., :d // 2]
    code = torch.stack((byte & 15, byte >> 4), -1).flatten(-2)
    exp, man = ((code >> 1) & 3).float(), (code & 1).float()
    mag = torch.where(exp > 0, (1.0 + 0.5 * man) * torch.exp2(exp - 1.0), 0.5 * man)
    value = torch.where(code >= 8, -mag, mag)
    scale = row[..., d // 2:].contiguous().view(torch.float8_e4m3fn).float()
    return (value.unflatten(-1, (-1, GROUP)) * scale[..., None]).flatten(-2)


def _store(x, dtype, scale):
    """fp32 values as a cache of the given type holds them."""
    if dtype == "fp4":
        return _pack(*_quantise(x / scale))
    if dtype == "fp8":
        return (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(TYPES[dtype])


def _values(row, dtype, d, scale):
    """Stored rows as fp32 values."""
    if dtype == "fp4":
        return _unpack(row, d) * scale
    if dtype == "fp8":
        return row.view(torch.float8_e4m3fn).float() * scale
    return row.float()


# -------------------------------------------------------------- the inputs

def _row_width(dtype, d):
    return d // 2 + d // GROUP if dtype == "fp4" else d


def _lengths(case):
    """The lengths of a case, evenly spread over its range (one sequence: the
    longest); the seed deals them out to the sequences."""
    lo, hi, b = case["ctx_min"], case["ctx_max"], case["batch"]
    return torch.tensor([hi - (hi - lo) * i // max(1, b - 1) for i in range(b)])


def _pages(case, gen, extra=0):
    """Ragged lengths, and a block table over shuffled pages (-1 = none)."""
    b = case["batch"]
    lens = _lengths(case)[torch.randperm(b, generator=gen)]
    nblk = (lens + PAGE - 1) // PAGE
    total = int(nblk.sum()) + extra
    perm = torch.randperm(total, generator=gen).int()
    table = torch.full((b, int(nblk.max())), -1, dtype=torch.int32)
    at = 0
    for i in range(b):
        n = int(nblk[i])
        table[i, :n] = perm[at:at + n]
        at += n
    return lens.int(), table, total, perm[at:]


def _cache(case, total, g, scale, dtype):
    """A cache of N(0, 1) values; a tenth of its channels are five times as
    large, as keys' channels are."""
    d, hkv = case["d"], case["hkv"]
    out = torch.empty((total, hkv, PAGE, _row_width(dtype, d)), device="cuda",
                      dtype=TYPES.get(dtype, torch.uint8))
    gain = 1.0 + 4.0 * (torch.rand((hkv, 1, d), device="cuda", generator=g) < 0.1)
    for at in range(0, total, 8192):
        n = min(8192, total - at)
        x = torch.randn((n, hkv, PAGE, d), device="cuda", generator=g) * gain
        out[at:at + n] = _store(x, dtype, scale)
    return out


def _tree_mask(q_len):
    """Ancestor bits of a binary tree in breadth-first order."""
    bits = [1]
    for c in range(1, q_len):
        bits.append(bits[(c - 1) // 2] | (1 << c))
    return torch.tensor(bits, dtype=torch.int32)


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, b, hkv, d = case["op"], case["batch"], case["hkv"], case["d"]
    dtype = case.get("dtype", "fp4")
    ks = float(case.get("k_scale", 1.0))
    if dtype == "fp8":
        ks = FP8_SCALE
    elif dtype in TYPES:
        ks = 1.0
    vs = ks if dtype == "fp8" or ks == 1.0 else 0.75 * ks
    io = TYPES.get(dtype, torch.bfloat16)
    extra = b * ((case["budget"] + PAGE - 1) // PAGE) if op == "evict" else 0
    lens, table, total, spare = _pages(case, gen, extra)
    s = dict(case=case, op=op, dtype=dtype, d=d, ks=ks, vs=vs,
             lens=lens.cuda(), table=table.cuda())
    s["k"] = _cache(case, total, g, ks, dtype)
    if op != "score":
        s["v"] = _cache(case, total, g, vs, dtype)
    if op == "append":
        n = case["n_new"]
        s["k_new"], s["v_new"] = (
            torch.randn((b, n, hkv, d), device="cuda", generator=g).to(io)
            for _ in range(2))
        return s
    if op == "evict":
        s["dst"] = spare.view(b, -1).contiguous().cuda()
        # summed softmax weights: a long tail, and keys never attended to
        w = torch.exp(2.0 * torch.randn((total, hkv, PAGE), device="cuda", generator=g))
        s["scores"] = torch.where(
            torch.rand(w.shape, device="cuda", generator=g) < 0.1, 0.0, w)
        return s
    hq, ql = case["hq"], case["q_len"]
    s["q"] = torch.randn((b, ql, hq, d), device="cuda", generator=g).to(io)
    s["scale"] = 1.0 / math.sqrt(d)
    s["tree"] = _tree_mask(ql).repeat(b, 1).cuda() if case["tree"] else None
    if op == "score":
        s["scores"] = torch.rand((total, hkv, PAGE), device="cuda", generator=g) * 4.0
        _, vis, x = _logits(s)
        s["lse"] = torch.logsumexp(x.masked_fill(~vis, -math.inf), -1).permute(
            0, 3, 1, 2).flatten(2).contiguous()
    return s


# --------------------------------------------------------- the plain forms

def _logical(cache, table):
    """Paged [nb, Hkv, 16, w] -> logical [B, Hkv, max_blocks * 16, w]."""
    return cache[table.clamp(min=0)].transpose(1, 2).flatten(2, 3)


def _visible(s, n):
    """[B, 1, 1, q_len, n]: the keys each query row attends to."""
    c = s["case"]
    ql = c["q_len"]
    j = torch.arange(n, device="cuda")
    i = torch.arange(ql, device="cuda")
    base = s["lens"].long()[:, None, None] - ql
    t = base + i[:, None]
    ok = j <= t
    if s["tree"] is not None:
        node = (j - base).clamp(0, 31)
        bit = (s["tree"].long()[:, :, None] >> node) & 1
        ok = ok & ((j < base) | (bit == 1))
    if c["window"]:
        ok = ok & ((j < c["n_sink"]) | (j > t - c["window"]))
    return ok[:, None, None]


def _logits(s):
    """Values of the valid keys [B, Hkv, 1, n, D], who sees them, and the
    scaled products [B, Hkv, group, q_len, n], fp32."""
    c = s["case"]
    n = s["table"].shape[1] * PAGE
    live = (torch.arange(n, device="cuda") < s["lens"][:, None])[:, None, :, None]
    k = _values(_logical(s["k"], s["table"]), s["dtype"], s["d"], s["ks"])
    k = torch.where(live, k, 0.0)
    q = s["q"].float().unflatten(2, (c["hkv"], -1)).permute(0, 2, 3, 1, 4)
    g = q.shape[2]
    x = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (g, -1))
    return live, _visible(s, n), x * s["scale"]


def _run_append(s):
    n = s["case"]["n_new"]
    pos = s["lens"].long()[:, None] - n + torch.arange(n, device="cuda")
    page = s["table"].gather(1, pos // PAGE).long()
    out = []
    for side, scale in (("k", s["ks"]), ("v", s["vs"])):
        s[side][page, :, pos % PAGE] = _store(s[side + "_new"].float(), s["dtype"], scale)
        got = s[side][page, :, pos % PAGE]
        got = _values(got, s["dtype"], s["d"], scale)
        out.append(got.to(s[side + "_new"].dtype))
    return out


def _run_attend(s):
    live, vis, x = _logits(s)
    v = _values(_logical(s["v"], s["table"]), s["dtype"], s["d"], s["vs"])
    v = torch.where(live, v, 0.0)
    x = x.masked_fill(~vis, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    g, ql = p.shape[2], p.shape[3]
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (g, ql)) / total
    lse = (m + torch.log(total))[..., 0]
    return (o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(s["q"].dtype).contiguous(),
            lse.permute(0, 3, 1, 2).flatten(2).contiguous())


def _run_score(s):
    c = s["case"]
    _, vis, x = _logits(s)
    lse = s["lse"].unflatten(2, (c["hkv"], -1)).permute(0, 2, 3, 1)[..., None]
    w = torch.exp(x - lse).masked_fill(~vis, 0.0).sum((2, 3))
    n = w.shape[-1]
    j = torch.arange(n, device="cuda")
    old = _logical(s["scores"][..., None], s["table"])[..., 0]
    new = j >= s["lens"][:, None, None] - c["q_len"]
    total = torch.where(new, 0.0, old) + w
    at = (j < s["lens"][:, None]).nonzero(as_tuple=True)
    page = s["table"][at[0], at[1] // PAGE].long()
    s["scores"][page, :, at[1] % PAGE] = total.transpose(1, 2)[at]
    return s["scores"]


def _run_evict(s):
    c = s["case"]
    budget, hkv = c["budget"], c["hkv"]
    lens = s["lens"].long()[:, None, None]
    old = _logical(s["scores"][..., None], s["table"])[..., 0]
    n = old.shape[-1]
    j = torch.arange(n, device="cuda")
    forced = (j < c["n_sink"]) | (j >= lens - c["n_recent"]) | (lens <= budget)
    rank = torch.where(forced, math.inf, old)
    rank = rank.masked_fill(j >= lens, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    kept = order[..., :budget]
    kept = torch.where(kept < lens, kept, n)
    kept = torch.sort(kept, dim=-1).values
    kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[-1]), value=n)
    b, h, slot = (kept < n).nonzero(as_tuple=True)
    pos = kept[b, h, slot]
    src = s["table"][b, pos // PAGE].long(), h, pos % PAGE
    dst = s["dst"][b, slot // PAGE].long(), h, slot % PAGE
    for side in ("k", "v", "scores"):
        s[side][dst] = s[side][src]
    kept = kept.masked_fill(kept >= n, -1).int()
    return _evicted(s, kept, s["lens"].clamp(max=budget))


def _evicted(s, kept, lens):
    """What an eviction leaves: positions, lengths, scores and the caches as
    values (a 4-bit cache through the rows of its destination pages)."""
    if s["dtype"] == "fp4":
        if own:
            import spec_verify_paged_gb300 as svp
            k, v = svp.kv_gather(s["k"], s["v"], s["dst"], lens, s["case"]["budget"],
                                 starts=torch.zeros_like(lens))
        else:
            live = torch.arange(s["case"]["budget"], device="cuda") < lens[:, None]
            k, v = (torch.where(live[:, :, None, None],
                                _unpack(_logical(s[x], s["dst"])[:, :, :live.shape[1]],
                                        s["d"]).transpose(1, 2), 0.0).to(torch.bfloat16)
                    for x in ("k", "v"))
        return kept, lens, s["scores"], k, v
    k, v = s["k"], s["v"]
    if s["dtype"] == "fp8":
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    return kept, lens, s["scores"], k, v


# ------------------------------------------------------ a user's own calls

def _own(s):
    import spec_verify_paged_gb300 as svp
    c = s["case"]
    if s["op"] == "append":
        svp.kv_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"],
                      s["lens"], k_scale=s["ks"], v_scale=s["vs"])
        return svp.kv_gather(s["k"], s["v"], s["table"], s["lens"], c["n_new"],
                             k_scale=s["ks"], v_scale=s["vs"])
    if s["op"] == "attend":
        if s["tree"] is not None:
            return svp.paged_tree_attention(
                s["q"], s["k"], s["v"], s["table"], s["lens"], s["tree"],
                scale=s["scale"], k_scale=s["ks"], v_scale=s["vs"])
        return svp.paged_decode_attention(
            s["q"], s["k"], s["v"], s["table"], s["lens"], n_sink=c["n_sink"],
            window=c["window"], scale=s["scale"], k_scale=s["ks"],
            v_scale=s["vs"])
    if s["op"] == "score":
        return svp.paged_score_update(
            s["q"], s["k"], s["lse"], s["table"], s["lens"], s["scores"],
            n_sink=c["n_sink"], window=c["window"], tree_mask=s["tree"],
            scale=s["scale"], k_scale=s["ks"])
    kept, lens = svp.kv_evict(
        s["k"], s["v"], s["scores"], s["table"], s["lens"], c["budget"],
        n_sink=c["n_sink"], n_recent=c["n_recent"], dst_block_table=s["dst"])
    return _evicted(s, kept, lens)


def run(s):
    if own:
        return _own(s)
    if s["op"] == "append":
        return _run_append(s)
    if s["op"] == "attend":
        return _run_attend(s)
    if s["op"] == "score":
        return _run_score(s)
    return _run_evict(s)


# ------------------------------------------------------------------- work

def _row_bytes(dtype, d):
    return {"fp4": d // 2 + d // GROUP, "fp8": d, "bf16": 2 * d, "f32": 4 * d}[dtype]


def work(case):
    op, b, hkv, d = case["op"], case["batch"], case["hkv"], case["d"]
    dtype = case.get("dtype", "fp4")
    row = _row_bytes(dtype, d)
    io = d * (4 if dtype == "f32" else 2)
    lens = _lengths(case).double()
    mean = float(lens.mean())
    if op == "append":
        rows = 2.0 * b * case["n_new"] * hkv
        # new rows in, cache rows out; the cache rows back as values
        return {"bytes": rows * (io + row) + rows * io, "flops": rows * d * 4.0}
    if op == "evict":
        kept = hkv * float(lens.clamp(max=case["budget"]).sum())
        moved = kept * (2 * row + 4)
        out = {"bytes": b * hkv * mean * 4.0 + 2.0 * moved + 4.0 * kept + 8.0 * b,
               "flops": b * hkv * mean * 2.0}
        if dtype == "fp4":
            out["bytes"] += 2.0 * kept * io
        return out
    hq, ql = case["hq"], case["q_len"]
    seen = mean
    if case["window"]:
        seen = float(lens.clamp(max=case["window"] + ql - 1 + case["n_sink"]).mean())
    sides = 2 if op == "attend" else 1
    io_bytes = b * ql * hq * (io * sides + 4.0)
    keep = b * hkv * seen * 8.0 if op == "score" else 0.0
    return {"bytes": sides * b * hkv * seen * row + io_bytes + keep,
            "flops": 2.0 * sides * b * ql * hq * d * seen}


# -------------------------------------------------- the definition, 64 bits

def _exact_rows(raw, dtype, d, scale):
    """Stored bytes as the values they stand for, float64."""
    if dtype in TYPES:
        return raw.double()
    byte = raw.int()

    def e4m3(u):
        exp, man = (u >> 3) & 15, u & 7
        mag = torch.where(exp > 0, (8 + man).double() * torch.exp2((exp - 10).double()),
                          man.double() * 2.0 ** -9)
        mag = torch.where((u & 127) == 127, math.nan, mag)
        return torch.where(u >= 128, -mag, mag)

    if dtype == "fp8":
        return e4m3(byte) * scale
    out = torch.empty(raw.shape[:-1] + (d,), dtype=torch.float64, device=raw.device)
    for half in (0, 1):
        u = (byte[..., :d // 2] >> (4 * half)) & 15
        exp, man = (u >> 1) & 3, u & 1
        mag = torch.where(exp > 0, (2 + man).double() * torch.exp2((exp - 2).double()),
                          0.5 * man.double())
        out[..., half::2] = torch.where(u >= 8, -mag, mag)
    step = e4m3(byte[..., d // 2:]).repeat_interleave(GROUP, -1)
    return out * step * scale


def _exact_store(x, dtype, scale):
    """The values a cache holds after the append of x, float64."""
    if dtype in TYPES:
        return x.double()
    y = (x.double() / scale).float().double()
    if dtype == "fp8":
        return y.clamp(-448, 448).float().to(torch.float8_e4m3fn).double() * scale
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    blocks = y.reshape(y.shape[:-1] + (-1, GROUP))
    big = (blocks.abs().amax(-1, keepdim=True) / 6).float().double().clamp(max=448)
    # E4M3 to nearest even: steps of 2^(e-3), e >= -6
    e = torch.floor(torch.log2(big.clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    sc = (torch.round(big / step) * step).clamp(2.0 ** -9, 448)
    r = (blocks.abs() / sc).float().double()
    best = torch.zeros_like(r)
    for i in range(1, 8):  # up to grid[i] from the midpoint on, ties to even
        mid = (grid[i - 1] + grid[i]) / 2
        best = torch.where((r > mid) | ((r == mid) & (i % 2 == 0)), grid[i], best)
    return (torch.sign(blocks) * best * sc).reshape(y.shape) * scale


def exact(case, seed):
    s = prepare(case, seed)
    op, d, dtype = case["op"], case["d"], s["dtype"]
    lens, table = s["lens"].tolist(), s["table"].cpu()
    if op == "append":
        return [_exact_store(s["k_new"], dtype, s["ks"]),
                _exact_store(s["v_new"], dtype, s["vs"])]
    if op == "evict":
        return _exact_evict(s, lens, table)
    b, hq, hkv, ql = case["batch"], case["hq"], case["hkv"], case["q_len"]
    per = hq // hkv
    out = torch.zeros((b, ql, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((b, ql, hq), dtype=torch.float64, device="cuda")
    scores = s["scores"].double() if op == "score" else None
    for i in range(b):
        n = lens[i]
        ids = table[i, :(n + PAGE - 1) // PAGE].long().cuda()
        see = torch.zeros((ql, n), dtype=torch.bool, device="cuda")
        for r in range(ql):
            t = n - ql + r
            see[r, :n - ql] = True
            for a in range(r + 1):
                see[r, n - ql + a] = (s["tree"] is None or
                                      bool((int(s["tree"][i, r]) >> a) & 1))
            if case["window"]:
                lo = max(0, t - case["window"] + 1)
                hidden = torch.arange(n, device="cuda")
                see[r] &= (hidden >= lo) | (hidden < case["n_sink"])
        for h in range(hkv):
            k = _exact_rows(s["k"][ids, h], dtype, d, s["ks"]).reshape(-1, d)[:n]
            q = s["q"][i, :, h * per:(h + 1) * per].double()
            x = torch.einsum("qhd,nd->qhn", q, k) * s["scale"]
            x = x.masked_fill(~see[:, None], -math.inf)
            if op == "score":
                w = torch.exp(x - s["lse"][i, :, h * per:(h + 1) * per, None].double())
                have = scores[ids, h].reshape(-1)
                have[n - ql:n] = 0.0
                have[:n] += w.sum((0, 1))
                scores[ids, h] = have.reshape(-1, PAGE)
                continue
            v = _exact_rows(s["v"][ids, h], dtype, d, s["vs"]).reshape(-1, d)[:n]
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            z = p.sum(-1, keepdim=True)
            out[i, :, h * per:(h + 1) * per] = torch.einsum("qhn,nd->qhd", p / z, v)
            lse[i, :, h * per:(h + 1) * per] = (top + torch.log(z))[..., 0]
    return scores if op == "score" else (out, lse)


def _exact_evict(s, lens, table):
    import numpy as np
    c = s["case"]
    budget, hkv, d, dtype = c["budget"], c["hkv"], s["d"], s["dtype"]
    scores, dst = s["scores"], s["dst"].cpu()
    kept = np.full((len(lens), hkv, budget), -1, np.int32)
    new_scores = scores.double()
    if dtype == "fp4":
        sides = [torch.zeros((len(lens), budget, hkv, d), dtype=torch.float64,
                             device="cuda") for _ in "kv"]
    else:
        raw = [s[x].view(torch.float8_e4m3fn).float() if dtype == "fp8" else s[x]
               for x in "kv"]
        sides = [x.clone() for x in raw]
    for i, n in enumerate(lens):
        ids = table[i, :(n + PAGE - 1) // PAGE].long()
        mine = scores[ids.cuda()].transpose(0, 1).reshape(hkv, -1)[:, :n].cpu().numpy()
        for h in range(hkv):
            if n <= budget:
                keep = np.arange(n)
            else:
                first, last = c["n_sink"], n - c["n_recent"]
                free = budget - c["n_sink"] - c["n_recent"]
                middle = np.argsort(-mine[h, first:last].astype(np.float64),
                                    kind="stable")[:free] + first
                keep = np.sort(np.concatenate((np.arange(first), middle,
                                               np.arange(last, n))))
            kept[i, h, :len(keep)] = keep
            at = torch.from_numpy(keep)
            to = torch.arange(len(keep))
            src = ids[at // PAGE].cuda(), (at % PAGE).cuda()
            out = dst[i, to // PAGE].long().cuda(), (to % PAGE).cuda()
            new_scores[out[0], h, out[1]] = scores[src[0], h, src[1]].double()
            for side, name in zip(range(2), "kv"):
                if dtype == "fp4":
                    rows = _exact_rows(s[name][src[0], h, src[1]], dtype, d, 1.0)
                    sides[side][i, :len(keep), h] = rows
                else:
                    sides[side][out[0], h, out[1]] = raw[side][src[0], h, src[1]]
    new_lens = torch.tensor([min(n, budget) for n in lens], dtype=torch.int32)
    return torch.from_numpy(kept), new_lens, new_scores, sides[0], sides[1]
