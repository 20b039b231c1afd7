"""Cases of page-sparse attention, page assignment and token log probabilities,
their plain forms and the calls a user makes of them.

Six operators of a speculative decoding step over long paged contexts (pages
of 16 positions, caches [num_blocks, Hkv, 16, row]):

  bounds    kv_page_bounds: per page and kv head the elementwise smallest and
            largest K, for the pages that hold a sequence's newest rows
  scores    paged_page_scores: from the bounds alone, what a query row's
            product with a key of the page can be at most, the largest over
            the query rows of the kv head
  select    paged_select_pages: the first pages, the newest and the best-scored
            others, a list per sequence and kv head
  sparse    paged_sparse_attention over the listed pages only
  assign    kv_assign_pages (pages taken for growing sequences, slots of the
            new rows), kv_append of the packed rows into those slots, and the
            pages released again
  logprobs  token_logprobs: log probability, rank and entropy of given tokens
            and the most likely alternatives

A 4-bit row of D elements is D/2 bytes of E2M1 codes (element 2i in the low
nibble of byte i) followed by D/16 E4M3 scales, one per 16 elements; an FP8 row
is D E4M3 codes.
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
        # after a decode step's append: one touched page per sequence and head,
        # the latency of one short launch
        dict(name="bounds step", op="bounds", dtype="bf16", batch=32, hkv=32,
             d=128, ctx_min=512, ctx_max=4096, n_new=1),
        # whole prompts that have just entered an FP8 cache
        dict(name="bounds prompt", op="bounds", dtype="fp8", batch=8, hkv=8,
             d=128, ctx_min=16384, ctx_max=65536, n_new=65536),
        # ordinary decode over long contexts, GQA group 4, one query position
        dict(name="scores decode", op="scores", dtype="bf16", batch=32, hq=32,
             hkv=8, d=128, q_len=1, ctx_min=8192, ctx_max=32768),
        # verification of 4 drafts and the bonus position over the longest
        # contexts: 40 query rows per kv head
        dict(name="scores verify", op="scores", dtype="bf16", batch=4, hq=64,
             hkv=8, d=128, q_len=5, ctx_min=131072, ctx_max=131072),
        # 2048 of up to 32,768 positions per sequence and head
        dict(name="select decode", op="select", batch=32, hkv=8,
             ctx_min=8192, ctx_max=32768, n_select=128, n_sink=1, n_recent=4),
        # 4096 of 131,072 positions
        dict(name="select long", op="select", batch=4, hkv=8, ctx_min=131072,
             ctx_max=131072, n_select=256, n_sink=1, n_recent=8),
        # decode over the selected pages of a bf16 cache
        dict(name="sparse decode", op="sparse", dtype="bf16", batch=32, hq=32,
             hkv=8, d=128, q_len=1, ctx_min=8192, ctx_max=32768, n_select=128,
             tree=False),
        # verification over the selected pages of an FP8 cache
        dict(name="sparse verify", op="sparse", dtype="fp8", batch=4, hq=64,
             hkv=8, d=128, q_len=5, ctx_min=131072, ctx_max=131072,
             n_select=256, tree=False),
        # a verification step's 5 rows get pages and slots, are stored, and the
        # drafts' pages go back
        dict(name="assign step", op="assign", dtype="bf16", batch=64, hkv=8,
             d=128, ctx_min=512, ctx_max=4096, new_min=5, new_max=5),
        # ragged prompts admitted to empty rows of the batch, and released
        dict(name="assign prompts", op="assign", dtype="bf16", batch=64, hkv=8,
             d=128, ctx_min=0, ctx_max=0, new_min=1, new_max=2048),
        # the tokens a verification emitted, with a few alternatives each
        dict(name="logprobs verify", op="logprobs", dtype="f32", rows=80,
             vocab=32000, n_top=5, temperature=1.0, padding=0.4, density=1.0),
        # many positions over a large vocabulary, constrained, 20 alternatives
        dict(name="logprobs many", op="logprobs", dtype="bf16", rows=512,
             vocab=131072, n_top=20, temperature=0.7, padding=0.0, density=0.9),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = max(work(c)["bytes"] for c in listed())
    flops = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(("bounds", "scores", "select", "sparse", "sparse",
                         "assign", "logprobs"))
        if op == "logprobs":
            c = dict(op=op, dtype=rng.choice(("f32", "bf16")),
                     rows=_log_int(rng, 1, 2048), vocab=_log_int(rng, 50, 200000),
                     n_top=rng.choice((0, 1, 2, 5, 5, 8, 20, 32)),
                     temperature=rng.choice((1.0, 1.0, 0.6, 1.7)),
                     padding=rng.choice((0.0, 0.0, 0.3)),
                     density=rng.choice((1.0, 1.0, 0.5, 0.02)))
            if work(c)["bytes"] <= top:
                return c
            continue
        hkv = rng.choice((1, 2, 3, 4, 8, 8, 16, 32))
        group = rng.choice((1, 1, 2, 3, 4, 4, 5, 7, 8))
        d = rng.choice((64, 128, 128))
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 40, 262144)
        lo = max(17, int(hi * rng.uniform(0.2, 1.0)))
        c = dict(op=op, batch=batch, hkv=hkv, d=d, ctx_min=lo, ctx_max=hi)
        pages = (hi + PAGE - 1) // PAGE
        n_select = min(2048, max(4, int(pages * rng.uniform(0.02, 1.1))))
        if op == "bounds":
            c.update(dtype=rng.choice(("bf16", "bf16", "fp8", "fp4", "f32")),
                     n_new=rng.choice((1, 5, 16, 17, 300, hi)))
        elif op == "scores":
            c.update(dtype=rng.choice(("bf16", "bf16", "f32")), hq=hkv * group,
                     q_len=rng.choice((1, 1, 2, 3, 5, 8, 16)))
        elif op == "select":
            del c["d"]
            c.update(n_select=n_select, n_sink=rng.randint(0, 2),
                     n_recent=rng.randint(0, n_select - 2))
        elif op == "sparse":
            c.update(dtype=rng.choice(("bf16", "bf16", "fp8", "fp4", "f32")),
                     hq=hkv * group, q_len=rng.choice((1, 1, 2, 3, 5, 8, 16)),
                     n_select=n_select, tree=rng.random() < 0.25)
        else:
            c["ctx_max"] = min(hi, 4096) if rng.random() < 0.7 else 0
            c["ctx_min"] = min(lo, c["ctx_max"])
            c.update(dtype=rng.choice(("bf16", "bf16", "fp8", "fp4", "f32")))
            c["new_max"] = _log_int(rng, 1, 4096)
            c["new_min"] = max(0, int(c["new_max"] * rng.uniform(-0.2, 1.0)))
        w = work(c)
        if w["bytes"] > top or w["flops"] > flops:
            continue
        # cached elements bound the memory of the inputs and the plain form
        cells = batch * (c["ctx_max"] + c.get("new_max", 0)) * hkv * d
        if op in ("bounds", "sparse", "assign") and cells > 700e6:
            continue
        if op == "scores" and batch * pages * hkv * (2 * d + group * c["q_len"]) > 1.2e9:
            continue
        if op == "sparse" and (batch * n_select * PAGE * hkv *
                               (2 * d + 2 * group * c["q_len"]) > 1.2e9):
            continue
        return c


# --------------------------------------------- the cache types, elementary

def _quantise(y):
    """fp32 y [..., D] -> 4-bit rows [..., D/2 + D/16] uint8."""
    blocks = y.unflatten(-1, (-1, GROUP))
    amax = blocks.abs().amax(-1)
    scale = (amax / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    scale = scale.clamp(min=2.0 ** -9)
    r = blocks.abs() / scale[..., None]
    code = ((r > 0.25).to(torch.uint8) + (r >= 0.75) + (r > 1.25) + (r >= 1.75) +
            (r > 2.5) + (r >= 3.5) + (r > 5.0))
    code = (code | (blocks < 0).to(torch.uint8) * 8).flatten(-2)
    byte = code[..., 0::2] | (code[..., 1::2] << 4)
    return torch.cat((byte, scale.to(torch.float8_e4m3fn).view(torch.uint8)), -1)


def _unpack(row, d):
    """4-bit rows -> code * scale, fp32 [..., D]."""
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
        return _quantise(x / scale)
    if dtype == "fp8":
        return (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(TYPES[dtype])


def _values(row, dtype, d):
    """Stored rows as fp32 values, before the cache's own scale factor."""
    if dtype == "fp4":
        return _unpack(row, d)
    if dtype == "fp8":
        return row.view(torch.float8_e4m3fn).float()
    return row.float()


# -------------------------------------------------------------- the inputs

def _spread(lo, hi, n):
    """n whole numbers evenly spread over [lo, hi], the largest first."""
    return torch.tensor([hi - (hi - lo) * i // max(1, n - 1) for i in range(n)])


def _lengths(case, gen):
    """The lengths of a case; the seed deals them out to the sequences."""
    lens = _spread(case["ctx_min"], case["ctx_max"], case["batch"])
    return lens[torch.randperm(case["batch"], generator=gen)]


def _pages(lens, gen, extra=0):
    """A block table over shuffled pages (-1 = none), the number of pages and
    `extra` pages that no sequence holds."""
    nblk = (lens + PAGE - 1) // PAGE
    total = int(nblk.sum()) + extra
    perm = torch.randperm(total, generator=gen).int()
    table = torch.full((len(lens), max(1, int(nblk.max()))), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(nblk.tolist()):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, total, perm[at:]


def _gain(hkv, d, g):
    """A tenth of the channels are five times as large, as keys' channels are."""
    return 1.0 + 4.0 * (torch.rand((hkv, 1, d), device="cuda", generator=g) < 0.1)


def _cache(case, total, g, scale, dtype):
    d, hkv = case["d"], case["hkv"]
    width = d // 2 + d // GROUP if dtype == "fp4" else d
    out = torch.empty((total, hkv, PAGE, width), device="cuda",
                      dtype=TYPES.get(dtype, torch.uint8))
    gain = _gain(hkv, d, g)
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


def _prepare_logprobs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, v = case["rows"], case["vocab"]
    s = dict(case=case, op=case["op"])
    logits = torch.empty((n, v), device="cuda", dtype=TYPES[case["dtype"]])
    for at in range(0, n, 256):
        m = min(256, n - at)
        logits[at:at + m] = 2.0 * torch.randn((m, v), device="cuda", generator=g)
    s["logits"] = logits
    s["allowed"] = None
    allow = torch.ones((1, 1), dtype=torch.bool, device="cuda")
    if case["density"] < 1.0:
        words = (v + 31) // 32
        allow = torch.rand((n, words * 32), device="cuda", generator=g) < case["density"]
        allow[:, v // 2] = True
        bit = torch.arange(32, device="cuda")
        packed = (allow.unflatten(-1, (words, 32)).long() << bit).sum(-1)
        s["allowed"] = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).int()
        allow = allow[:, :v]
    # the tokens are drawn from the rows' distributions
    tokens = torch.empty(n, dtype=torch.int32, device="cuda")
    for at in range(0, n, 256):
        z = logits[at:at + 256].float() / case["temperature"]
        z = z.masked_fill(~allow[at:at + 256] if allow.shape[0] > 1 else ~allow, -math.inf)
        u = torch.rand(z.shape, device="cuda", generator=g).clamp(min=1e-9)
        tokens[at:at + 256] = (z - torch.log(-torch.log(u))).argmax(-1).int()
    pad = torch.rand(n, device="cuda", generator=g) < case["padding"]
    s["tokens"] = tokens.masked_fill(pad, -1)
    return s


def prepare(case, seed):
    if case["op"] == "logprobs":
        return _prepare_logprobs(case, seed)
    gen = torch.Generator().manual_seed(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, b, hkv = case["op"], case["batch"], case["hkv"]
    lens = _lengths(case, gen)
    s = dict(case=case, op=op, lens=lens.int().cuda())
    if op == "select":
        n = (case["ctx_max"] + PAGE - 1) // PAGE
        x = 10.0 + 5.0 * torch.randn((b, hkv, n), device="cuda", generator=g)
        x = torch.round(x * 4096.0) / 4096.0  # some scores are equal
        none = torch.arange(n, device="cuda") * PAGE >= s["lens"][:, None]
        s["scores"] = x.masked_fill(none[:, None], -math.inf)
        return s
    d, dtype = case["d"], case["dtype"]
    scale = {"fp8": FP8_SCALE, "fp4": 0.0371}.get(dtype, 1.0)
    s.update(dtype=dtype, d=d, ks=scale, vs=scale)
    io = TYPES.get(dtype, torch.bfloat16)
    if op == "assign":
        new = _spread(case["new_min"], case["new_max"], b)
        new = new[torch.randperm(b, generator=gen)]
        grown = lens + new
        more = int(((grown + PAGE - 1) // PAGE - (lens + PAGE - 1) // PAGE).sum())
        table, total, spare = _pages(lens, gen, more + 16)
        wide = torch.full((b, int(((grown + PAGE - 1) // PAGE).max()) + 1), -1,
                          dtype=torch.int32)
        wide[:, :table.shape[1]] = table[:, :wide.shape[1]]
        rows = int(new.sum())
        s.update(table=wide.cuda(), old=lens.int().cuda(), new=grown.int().cuda(),
                 free=spare.cuda(), rows=rows,
                 count=torch.tensor([len(spare)], dtype=torch.int32).cuda())
        shape = (total, hkv, PAGE, d // 2 + d // GROUP if dtype == "fp4" else d)
        s["k"], s["v"] = (torch.zeros(shape, device="cuda",
                                      dtype=TYPES.get(dtype, torch.uint8))
                          for _ in range(2))
        s["k_new"], s["v_new"] = (
            torch.randn((rows, hkv, d), device="cuda", generator=g).to(io)
            for _ in range(2))
        return s
    table, total, _ = _pages(lens, gen)
    s["table"] = table.cuda()
    if op == "bounds":
        s["k"] = _cache(case, total, g, scale, dtype)
        s["bounds"] = torch.zeros((total, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
        return s
    hq, ql = case["hq"], case["q_len"]
    s["q"] = torch.randn((b, ql, hq, d), device="cuda", generator=g).to(io)
    s["scale"] = 1.0 / math.sqrt(d)
    if op == "scores":
        # 16 keys spread by about 1.8 around the page's mean
        gain = _gain(hkv, d, g)
        mid = 0.5 * torch.randn((total, hkv, 1, d), device="cuda", generator=g)
        half = 1.3 + 0.9 * torch.rand((total, hkv, 1, d), device="cuda", generator=g)
        s["bounds"] = (torch.cat((mid - half, mid + half), 2) * gain).to(torch.bfloat16)
        return s
    s["k"] = _cache(case, total, g, scale, dtype)
    s["v"] = _cache(case, total, g, scale, dtype)
    s["tree"] = _tree_mask(ql).repeat(b, 1).cuda() if case["tree"] else None
    # the first page, the newest three and a random rest, in order
    n = (s["lens"].long() + PAGE - 1) // PAGE
    j = torch.arange(table.shape[1], device="cuda")
    rank = torch.rand((b, hkv, len(j)), device="cuda", generator=g)
    last = n[:, None, None]
    rank = rank.masked_fill((j == 0) | (j >= last - 3), 2.0).masked_fill(j >= last, -1.0)
    take = min(case["n_select"], len(j))
    best, at = torch.sort(rank, dim=-1, descending=True)
    at = at[..., :take].masked_fill(best[..., :take] < 0, 1 << 30)
    at = torch.sort(at, dim=-1).values
    at = at.masked_fill(at == 1 << 30, -1).int()
    s["pages"] = torch.nn.functional.pad(at, (0, case["n_select"] - take), value=-1)
    return s


# --------------------------------------------------------- the plain forms

def _outward(x, up):
    """fp32 x as the nearest bf16 value that is not smaller (up) or larger."""
    bits = x.view(torch.int32)
    cut = bits & -65536
    away = (cut != bits) & ((x > 0) if up else (x < 0))
    return (cut + away.int() * 65536).view(torch.float32).to(torch.bfloat16)


def _run_bounds(s):
    c = s["case"]
    n = (s["lens"].long() + PAGE - 1) // PAGE
    j = torch.arange(s["table"].shape[1], device="cuda")
    first = (s["lens"].long() - c["n_new"]).clamp(min=0) // PAGE
    touched = (j >= first[:, None]) & (j < n[:, None])
    b, p = touched.nonzero(as_tuple=True)
    for at in range(0, len(b), 16384):
        bb, pp = b[at:at + 16384], p[at:at + 16384]
        page = s["table"][bb, pp].long()
        k = _values(s["k"][page], s["dtype"], s["d"])
        pos = pp[:, None] * PAGE + torch.arange(PAGE, device="cuda")
        live = (pos < s["lens"][bb][:, None])[:, None, :, None]
        lo = torch.where(live, k, math.inf).amin(2)
        hi = torch.where(live, k, -math.inf).amax(2)
        s["bounds"][page] = torch.stack((_outward(lo, False), _outward(hi, True)), 2)
    return s["bounds"]


def _run_scores(s):
    c = s["case"]
    q = s["q"].float().unflatten(2, (c["hkv"], -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    b = s["bounds"][s["table"].clamp(min=0).long()].transpose(1, 2).float()
    x = torch.matmul(q.clamp(min=0.0), b[..., 1, :].transpose(-1, -2))
    x = x + torch.matmul(q.clamp(max=0.0), b[..., 0, :].transpose(-1, -2))
    x = x.amax(2) * s["scale"]
    none = torch.arange(x.shape[-1], device="cuda") * PAGE >= s["lens"][:, None]
    return x.masked_fill(none[:, None], -math.inf)


def _run_select(s):
    c = s["case"]
    x = s["scores"]
    n = ((s["lens"].long() + PAGE - 1) // PAGE)[:, None, None]
    j = torch.arange(x.shape[-1], device="cuda")
    forced = (j < c["n_sink"]) | (j >= n - c["n_recent"])
    rank = torch.where(forced, math.inf, x).masked_fill(j >= n, -math.inf)
    kept = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    kept = kept[..., :c["n_select"]]
    none = 1 << 30
    kept = torch.sort(torch.where(kept < n, kept, none), dim=-1).values
    kept = kept.masked_fill(kept == none, -1)
    kept = torch.nn.functional.pad(kept, (0, c["n_select"] - kept.shape[-1]), value=-1)
    return kept.int()


def _run_sparse(s):
    c = s["case"]
    ql, hkv = c["q_len"], c["hkv"]
    pages = s["pages"].long()
    bi = torch.arange(c["batch"], device="cuda")[:, None, None]
    hi = torch.arange(hkv, device="cuda")[None, :, None]
    phys = s["table"].long()[bi, pages.clamp(min=0)]
    k = _values(s["k"][phys, hi], s["dtype"], s["d"]).flatten(2, 3) * s["ks"]
    v = _values(s["v"][phys, hi], s["dtype"], s["d"]).flatten(2, 3) * s["vs"]
    pos = (pages[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(2)
    lens = s["lens"].long()[:, None, None]
    live = (pos >= 0) & (pos < lens)                          # [B, Hkv, n]
    k, v = (torch.where(live[..., None], x, 0.0) for x in (k, v))
    base = lens[..., None] - ql                               # [B, 1, 1, 1]
    row = torch.arange(ql, device="cuda")[:, None]
    seen = live[:, :, None] & (pos[:, :, None] <= base + row)  # [B, Hkv, q_len, n]
    if s["tree"] is not None:
        node = (pos[:, :, None] - base).clamp(0, 31)
        bit = (s["tree"].long()[:, None, :, None] >> node) & 1
        seen = seen & ((pos[:, :, None] < base) | (bit == 1))
    q = s["q"].float().unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4)
    g = q.shape[3]
    x = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)) * s["scale"]
    x = x.unflatten(2, (ql, g)).masked_fill(~seen[:, :, :, None], -math.inf).flatten(2, 3)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = (torch.matmul(p, v) / total).unflatten(2, (ql, g))
    lse = (m + torch.log(total))[..., 0].unflatten(2, (ql, g))
    return (o.permute(0, 2, 1, 3, 4).flatten(2, 3).to(s["q"].dtype).contiguous(),
            lse.permute(0, 2, 1, 3).flatten(2).contiguous())


def _plain_assign(s, target, want_slots):
    """Pages for the target lengths: those past them go onto the stack of free
    pages in order, those missing are taken from its top in order."""
    table, free = s["table"], s["free"]
    lens, new = s["lens"].long(), target.long()
    have, want = (lens + PAGE - 1) // PAGE, (new + PAGE - 1) // PAGE
    j = torch.arange(table.shape[1], device="cuda")
    gone = (j >= want[:, None]) & (j < have[:, None])
    back = table[gone]
    at = s["count"].long() + torch.arange(len(back), device="cuda")
    free[at] = back
    table[gone] = -1
    top = s["count"].long() + len(back)
    miss = (j >= have[:, None]) & (j < want[:, None])
    n = int(miss.sum())
    table[miss] = free[top - 1 - torch.arange(n, device="cuda")]
    s["count"].copy_(top - n)
    s["lens"].copy_(new)
    if not want_slots:
        return None, None
    more = (new - lens).clamp(min=0)
    offsets = torch.nn.functional.pad(torch.cumsum(more, 0), (1, 0))
    seq = torch.repeat_interleave(torch.arange(len(more), device="cuda"), more)
    pos = lens[seq] + torch.arange(len(seq), device="cuda") - offsets[seq]
    slots = table[seq, pos // PAGE].long() * PAGE + pos % PAGE
    return slots, offsets.int()


def _run_assign(s):
    slots, offsets = _plain_assign(s, s["new"], True)
    for side, scale in (("k", s["ks"]), ("v", s["vs"])):
        s[side][slots // PAGE, :, slots % PAGE] = _store(
            s[side + "_new"].float(), s["dtype"], scale)
    _plain_assign(s, s["old"], False)
    return _assigned(s, slots, offsets)


def _assigned(s, slots, offsets):
    """What the calls leave, the caches as the values they stand for."""
    k, v = s["k"], s["v"]
    if s["dtype"] == "fp8":
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    elif s["dtype"] == "fp4":
        k, v = _unpack(k, s["d"]), _unpack(v, s["d"])
    return slots, offsets, s["table"], s["lens"], s["free"], s["count"], k, v


def _allowed(s, at, n):
    v = s["case"]["vocab"]
    if s["allowed"] is None:
        return torch.ones((1, v), dtype=torch.bool, device="cuda")
    bit = torch.arange(32, device="cuda")
    return ((s["allowed"][at:at + n, :, None] >> bit) & 1).bool().flatten(1)[:, :v]


def _run_logprobs(s):
    c = s["case"]
    n, v, top = c["rows"], c["vocab"], c["n_top"]
    logp = torch.zeros(n, device="cuda")
    entropy = torch.zeros(n, device="cuda")
    rank = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    best = torch.full((n, top), -math.inf, device="cuda")
    which = torch.full((n, top), -1, dtype=torch.int32, device="cuda")
    for at in range(0, n, 128):
        m = min(128, n - at)
        token = s["tokens"][at:at + m].long()
        real = token >= 0
        x = s["logits"][at:at + m].float().masked_fill(~_allowed(s, at, m), -math.inf)
        z = x / c["temperature"]
        peak = z.amax(-1, keepdim=True)
        e = torch.exp(z - peak)
        total = e.sum(-1)
        lse = peak[:, 0] + torch.log(total)
        gap = torch.where(e > 0, z - peak, 0.0)
        mine = x.gather(1, token.clamp(min=0)[:, None])
        j = torch.arange(v, device="cuda")
        ahead = (x > mine) | ((x == mine) & (j < token[:, None]))
        logp[at:at + m] = torch.where(
            real, z.gather(1, token.clamp(min=0)[:, None])[:, 0] - lse, 0.0)
        entropy[at:at + m] = torch.where(
            real, torch.log(total) - (e * gap).sum(-1) / total, 0.0)
        rank[at:at + m] = torch.where(real, ahead.sum(-1), -1).int()
        if top:
            val, idx = torch.sort(x, dim=-1, descending=True, stable=True)
            k = min(top, v)
            val, idx = val[:, :k], idx[:, :k]
            some = (val > -math.inf) & real[:, None]
            best[at:at + m, :k] = torch.where(
                some, val / c["temperature"] - lse[:, None], -math.inf)
            which[at:at + m, :k] = torch.where(some, idx, -1).int()
    return logp, entropy, rank, best, which


# ------------------------------------------------------ a user's own calls

def _own(s):
    import spec_verify_paged_gb300 as svp
    c, op = s["case"], s["op"]
    if op == "bounds":
        return svp.kv_page_bounds(s["k"], s["table"], s["lens"], s["bounds"],
                                  n_new=c["n_new"])
    if op == "scores":
        return svp.paged_page_scores(s["q"], s["bounds"], s["table"], s["lens"],
                                     scale=s["scale"])
    if op == "select":
        return svp.paged_select_pages(s["scores"], s["lens"], c["n_select"],
                                      n_sink=c["n_sink"], n_recent=c["n_recent"])
    if op == "sparse":
        return svp.paged_sparse_attention(
            s["q"], s["k"], s["v"], s["table"], s["lens"], s["pages"],
            tree_mask=s["tree"], scale=s["scale"], k_scale=s["ks"],
            v_scale=s["vs"])
    if op == "assign":
        slots, offsets = svp.kv_assign_pages(
            s["table"], s["lens"], s["new"], s["free"], s["count"],
            n_slots=s["rows"])
        svp.kv_append(s["k_new"], s["v_new"], s["k"], s["v"], slots=slots,
                      k_scale=s["ks"], v_scale=s["vs"])
        svp.kv_assign_pages(s["table"], s["lens"], s["old"], s["free"], s["count"])
        return _assigned(s, slots, offsets)
    return svp.token_logprobs(s["logits"], s["tokens"], n_top=c["n_top"],
                              temperature=c["temperature"], allowed=s["allowed"])


def run(s):
    if own:
        return _own(s)
    return {"bounds": _run_bounds, "scores": _run_scores, "select": _run_select,
            "sparse": _run_sparse, "assign": _run_assign,
            "logprobs": _run_logprobs}[s["op"]](s)


# ------------------------------------------------------------------- work

def _row_bytes(dtype, d):
    return {"fp4": d // 2 + d // GROUP, "fp8": d, "bf16": 2 * d, "f32": 4 * d}[dtype]


def work(case):
    op = case["op"]
    if op == "logprobs":
        n = case["rows"] * (1.0 - case["padding"])
        size = 4 if case["dtype"] == "f32" else 2
        mask = case["vocab"] / 8.0 if case["density"] < 1.0 else 0.0
        out = case["rows"] * (16.0 + 8.0 * case["n_top"])
        return {"bytes": n * (case["vocab"] * size + mask) + out,
                "flops": n * case["vocab"] * 6.0}
    b, hkv = case["batch"], case["hkv"]
    lens = _spread(case["ctx_min"], case["ctx_max"], b).double()
    pages = torch.ceil(lens / PAGE)
    if op == "select":
        out = b * hkv * case["n_select"] * 4.0
        return {"bytes": hkv * float(pages.sum()) * 4.0 + out,
                "flops": hkv * float(pages.sum()) * 2.0}
    d, dtype = case["d"], case["dtype"]
    row = _row_bytes(dtype, d)
    io = d * (4 if dtype == "f32" else 2)
    if op == "bounds":
        first = torch.floor((lens - case["n_new"]).clamp(min=0) / PAGE)
        rows = hkv * float((lens - first * PAGE).sum())
        out = hkv * float((pages - first).sum()) * 4.0 * d
        return {"bytes": rows * row + out, "flops": rows * d * 2.0}
    if op == "scores":
        n = hkv * float(pages.sum())
        rows = case["hq"] // hkv * case["q_len"]
        return {"bytes": n * (4.0 * d + 4.0) + b * hkv * rows * io,
                "flops": n * rows * 4.0 * d}
    if op == "sparse":
        seen = hkv * float(torch.minimum(lens, pages.clamp(max=case["n_select"]) * PAGE).sum())
        rows = case["hq"] // hkv * case["q_len"]
        return {"bytes": seen * 2.0 * row + b * hkv * rows * (2.0 * io + 4.0) +
                b * hkv * case["n_select"] * 4.0,
                "flops": seen * rows * 4.0 * d}
    new = _spread(case["new_min"], case["new_max"], b).double()
    rows = float(new.sum())
    moved = rows / PAGE + b
    # rows in and stored, their slots, the pages' table entries and stack
    # entries taken and given back
    return {"bytes": rows * (hkv * 2.0 * (io + row) + 8.0) + moved * 16.0 + b * 24.0,
            "flops": rows * hkv * d * 2.0}


# -------------------------------------------------- the definition, 64 bits

def _exact_rows(raw, dtype, d):
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
        return e4m3(byte)
    out = torch.empty(raw.shape[:-1] + (d,), dtype=torch.float64, device=raw.device)
    for half in (0, 1):
        u = (byte[..., :d // 2] >> (4 * half)) & 15
        exp, man = (u >> 1) & 3, u & 1
        mag = torch.where(exp > 0, (2 + man).double() * torch.exp2((exp - 2).double()),
                          0.5 * man.double())
        out[..., half::2] = torch.where(u >= 8, -mag, mag)
    step = e4m3(byte[..., d // 2:]).repeat_interleave(GROUP, -1)
    return out * step


def _exact_store(x, dtype, scale):
    """The values (before the scale factor) a cache holds of x, float64."""
    if dtype in TYPES:
        return x.double()
    y = (x.double() / scale).float().double()
    if dtype == "fp8":
        return y.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    blocks = y.reshape(y.shape[:-1] + (-1, 16))
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
    return (torch.sign(blocks) * best * sc).reshape(y.shape)


def _exact_bounds(s):
    c = s["case"]
    d, dtype = s["d"], s["dtype"]
    out = s["bounds"].double()

    def grid(x):  # the step of bf16 values of x's magnitude
        e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -126)))
        return torch.exp2(e - 7)

    for b, n in enumerate(s["lens"].tolist()):
        first = max(0, n - c["n_new"]) // PAGE
        last = (n + PAGE - 1) // PAGE
        for p0 in range(first, last, 2048):
            p1 = min(last, p0 + 2048)
            ids = s["table"][b, p0:p1].long()
            k = _exact_rows(s["k"][ids], dtype, d)
            lo, hi = k.amin(2), k.amax(2)
            if p1 == last and n % PAGE:
                lo[-1], hi[-1] = (f(k[-1, :, :n % PAGE], 1) for f in (torch.amin, torch.amax))
            out[ids, :, 0] = torch.floor(lo / grid(lo)) * grid(lo)
            out[ids, :, 1] = torch.ceil(hi / grid(hi)) * grid(hi)
    return out


def _exact_scores(s):
    c = s["case"]
    per = c["hq"] // c["hkv"]
    b, n = s["table"].shape
    out = torch.full((b, c["hkv"], n), -math.inf, dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["lens"].tolist()):
        m = (length + PAGE - 1) // PAGE
        ids = s["table"][i, :m].long()
        for h in range(c["hkv"]):
            lo, hi = s["bounds"][ids, h].double().unbind(1)
            for r in range(c["q_len"]):
                for a in range(per):
                    q = s["q"][i, r, h * per + a].double() * s["scale"]
                    most = torch.where(q > 0, hi * q, lo * q).sum(-1)
                    out[i, h, :m] = torch.maximum(out[i, h, :m], most)
    return out


def _exact_select(s):
    import numpy as np
    c = s["case"]
    x = s["scores"].cpu().numpy().astype(np.float64)
    out = np.full((c["batch"], c["hkv"], c["n_select"]), -1, np.int32)
    for i, length in enumerate(s["lens"].tolist()):
        n = -(-length // PAGE)
        for h in range(c["hkv"]):
            if n <= c["n_select"]:
                out[i, h, :n] = np.arange(n)
                continue
            first, last = c["n_sink"], n - c["n_recent"]
            free = c["n_select"] - c["n_sink"] - c["n_recent"]
            middle = np.argsort(-x[i, h, first:last], kind="stable")[:free] + first
            out[i, h] = np.sort(np.concatenate(
                (np.arange(first), middle, np.arange(last, n))))
    return torch.from_numpy(out)


def _exact_sparse(s):
    c = s["case"]
    ql, per, d = c["q_len"], c["hq"] // c["hkv"], s["d"]
    out = torch.zeros((c["batch"], ql, c["hq"], d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((c["batch"], ql, c["hq"]), dtype=torch.float64, device="cuda")
    lists = s["pages"].tolist()
    offset = torch.arange(PAGE, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        for h in range(c["hkv"]):
            page = torch.tensor([p for p in lists[i][h] if p >= 0], device="cuda")
            pos = (page[:, None] * PAGE + offset).flatten()
            ids = s["table"][i].long()[page]
            keep = pos < n
            pos = pos[keep]
            k = _exact_rows(s["k"][ids, h], s["dtype"], d).reshape(-1, d)[keep] * s["ks"]
            v = _exact_rows(s["v"][ids, h], s["dtype"], d).reshape(-1, d)[keep] * s["vs"]
            see = torch.zeros((ql, len(pos)), dtype=torch.bool, device="cuda")
            for r in range(ql):
                see[r] = pos < n - ql
                for a in range(r + 1):
                    if s["tree"] is None or (int(s["tree"][i, r]) >> a) & 1:
                        see[r] |= pos == n - ql + a
            q = s["q"][i, :, h * per:(h + 1) * per].double()
            x = torch.einsum("qhd,nd->qhn", q, k) * s["scale"]
            x = x.masked_fill(~see[:, None], -math.inf)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            z = p.sum(-1, keepdim=True)
            out[i, :, h * per:(h + 1) * per] = torch.einsum("qhn,nd->qhd", p / z, v)
            lse[i, :, h * per:(h + 1) * per] = (top + torch.log(z))[..., 0]
    return out, lse


def _exact_assign(s):
    table = [[p for p in row if p >= 0] for row in s["table"].tolist()]
    width = s["table"].shape[1]
    stack = s["free"].tolist()
    height = len(stack)
    slots, offsets = [], [0]
    old, new = s["old"].tolist(), s["new"].tolist()
    for i, (a, b) in enumerate(zip(old, new)):
        while len(table[i]) * PAGE < b:
            height -= 1
            table[i].append(stack[height])
        slots += [table[i][p // PAGE] * PAGE + p % PAGE for p in range(a, b)]
        offsets.append(len(slots))
    for i, a in enumerate(old):
        keep = (a + PAGE - 1) // PAGE
        for page in table[i][keep:]:
            stack[height] = page
            height += 1
        table[i] = table[i][:keep] + [-1] * (width - keep)
    slots = torch.tensor(slots, dtype=torch.int64)
    sides = []
    for side, scale in (("k", s["ks"]), ("v", s["vs"])):
        value = _exact_rows(s[side], s["dtype"], s["d"])
        at = slots.cuda()
        value[at // PAGE, :, at % PAGE] = _exact_store(s[side + "_new"], s["dtype"], scale)
        sides.append(value)
    return (slots, torch.tensor(offsets, dtype=torch.int32),
            torch.tensor(table, dtype=torch.int32), s["old"],
            torch.tensor(stack, dtype=torch.int32),
            torch.tensor([height], dtype=torch.int32), *sides)


def _exact_logprobs(s):
    import numpy as np
    c = s["case"]
    n, v, top = c["rows"], c["vocab"], c["n_top"]
    logp, entropy = np.zeros(n), np.zeros(n)
    rank = np.full(n, -1, np.int32)
    best, which = np.full((n, top), -np.inf), np.full((n, top), -1, np.int32)
    for i, t in enumerate(s["tokens"].tolist()):
        if t < 0:
            continue
        x = s["logits"][i].double().cpu().numpy()
        ids = np.arange(v)
        if s["allowed"] is not None:
            bits = s["allowed"][i].cpu().numpy().view(np.uint8)
            ids = ids[np.unpackbits(bits, bitorder="little")[:v] > 0]
        x = x[ids]
        z = x / c["temperature"]
        p = np.exp(z - z.max())
        total = p.sum()
        lse = z.max() + np.log(total)
        p /= total
        mine = x[ids == t][0]
        logp[i] = mine / c["temperature"] - lse
        entropy[i] = -(p[p > 0] * (z[p > 0] - lse)).sum()
        rank[i] = (x > mine).sum() + ((x == mine) & (ids < t)).sum()
        if top:
            edge = np.partition(x, max(0, len(x) - top))[max(0, len(x) - top)]
            some = np.nonzero(x >= edge)[0]
            order = some[np.argsort(-x[some], kind="stable")][:top]
            best[i, :len(order)] = z[order] - lse
            which[i, :len(order)] = ids[order]
    return (torch.from_numpy(logp), torch.from_numpy(entropy), torch.from_numpy(rank),
            torch.from_numpy(best), torch.from_numpy(which))


def exact(case, seed):
    s = prepare(case, seed)
    return {"bounds": _exact_bounds, "scores": _exact_scores,
            "select": _exact_select, "sparse": _exact_sparse,
            "assign": _exact_assign, "logprobs": _exact_logprobs}[s["op"]](s)
