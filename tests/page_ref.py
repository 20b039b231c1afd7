"""Plain 64-bit forms of page bounds, page scores, page selection, attention
over listed pages, page assignment and token log probabilities (numpy and
lists, loops over sequences and heads)."""
import numpy as np

from cache_ref import PAGE, visible


def bf16_outward(x, up):
    """float64 -> the nearest bf16 value that is not smaller (up) or larger."""
    with np.errstate(invalid="ignore"):
        e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126)))
        step = 2.0 ** (e - 7)
        r = (np.ceil if up else np.floor)(x / step) * step
    return np.where(np.isfinite(x), r, x)


def bounds(values, lens, table, n_new, old):
    """values [nb, Hkv, 16, D] float64; old [nb, Hkv, 2, D]: a copy with the
    touched pages' bounds."""
    out = old.copy()
    for b, n in enumerate(lens):
        for p in range(max(0, int(n) - n_new) // PAGE, -(-int(n) // PAGE)):
            rows = values[table[b, p], :, :min(PAGE, int(n) - p * PAGE)]
            out[table[b, p], :, 0] = bf16_outward(rows.min(1), False)
            out[table[b, p], :, 1] = bf16_outward(rows.max(1), True)
    return out


def scores(q, bnd, lens, table, scale):
    """[B, Hkv, width], and the magnitude sum |q| max(|lo|, |hi|) |scale| that
    the error of a sum is relative to (the largest over the rows)."""
    B, ql, hq, d = q.shape
    hkv = bnd.shape[1]
    per = hq // hkv
    out = np.full((B, hkv, table.shape[1]), -np.inf)
    mag = np.zeros(out.shape)
    for b in range(B):
        for p in range(-(-int(lens[b]) // PAGE)):
            for h in range(hkv):
                lo, hi = bnd[table[b, p], h]
                x = q[b, :, h * per:(h + 1) * per].reshape(-1, d) * np.sign(scale)
                with np.errstate(invalid="ignore"):
                    s = (np.maximum(x, 0) * hi + np.minimum(x, 0) * lo).sum(-1)
                out[b, h, p] = s.max() * abs(scale)
                mag[b, h, p] = (np.abs(x) * np.maximum(np.abs(lo), np.abs(hi))
                                ).sum(-1).max() * abs(scale)
    return out, mag


def select(sc, lens, n_select, n_sink, n_recent):
    B, H, _ = sc.shape
    out = np.full((B, H, n_select), -1, np.int32)
    for b in range(B):
        n = -(-int(lens[b]) // PAGE)
        for h in range(H):
            if n <= n_select:
                out[b, h, :n] = np.arange(n)
                continue
            x = sc[b, h].astype(np.float64)
            x = np.where(np.isnan(x), np.inf, x)
            first = np.isnan(sc[b, h])  # NaN above +inf
            mid = np.arange(n_sink, n - n_recent)
            order = np.lexsort((mid, -x[mid], ~first[mid]))
            best = mid[order[:n_select - n_sink - n_recent]]
            out[b, h] = np.sort(np.concatenate(
                [np.arange(n_sink), best, np.arange(n - n_recent, n)]))
    return out


def sparse_attention(q, k, v, scale, lens, table, pages, tree=None):
    """out, lse and, per row, the largest sum|q||k| |scale| and max|v| over the
    keys it sees.  A page listed twice counts twice."""
    B, ql, hq, d = q.shape
    per = hq // k.shape[1]
    out, lse = np.zeros((B, ql, hq, d)), np.full((B, ql, hq), -np.inf)
    mag, vmax = np.zeros((B, ql, hq)), np.zeros((B, ql, hq))
    for b in range(B):
        L = int(lens[b])
        for h in range(hq):
            g = h // per
            pos = [p * PAGE + r for p in pages[b, g] if p >= 0
                   for r in range(PAGE) if p * PAGE + r < L]
            pos = np.array(pos, int)
            kk = k[table[b, pos // PAGE], g, pos % PAGE]
            vv = v[table[b, pos // PAGE], g, pos % PAGE]
            for i in range(ql):
                ok = visible(L, ql, i, 0, 0, None if tree is None else tree[b])[pos]
                if not ok.any():
                    continue
                x = kk[ok] @ q[b, i, h] * scale
                m = x.max()
                p = np.exp(x - m)
                out[b, i, h] = p @ vv[ok] / p.sum()
                lse[b, i, h] = m + np.log(p.sum())
                mag[b, i, h] = (np.abs(kk[ok]) @ np.abs(q[b, i, h])).max() * abs(scale)
                vmax[b, i, h] = np.abs(vv[ok]).max()
    return out, lse, mag, vmax


def assign(table, lens, new, stack, count, n_slots=None, num_blocks=2 ** 31 - 1):
    """The state after the call, (table, lens, stack, count, slots, offsets) of
    copies, and whether something was not served."""
    table, lens, stack = table.copy(), lens.copy(), stack.copy()
    B, width = table.shape
    cap = width * PAGE
    none = [-1] * (n_slots or 0)
    good = [0 <= lens[b] <= cap and 0 <= new[b] <= cap for b in range(B)]
    have = [-(-int(lens[b]) // PAGE) for b in range(B)]
    want = [-(-int(new[b]) // PAGE) for b in range(B)]
    back = sum(max(0, have[b] - want[b]) for b in range(B) if good[b])
    if count < 0 or count + back > len(stack):
        return table, lens, stack, count, none, [0] * (B + 1), True
    for b in range(B):
        if good[b]:
            for p in range(want[b], have[b]):
                stack[count] = table[b, p]
                table[b, p] = -1
                count += 1
    slots, offsets, short, asked = [], [0], False, 0
    full = False
    room = count
    for b in range(B):
        rows = max(0, int(new[b]) - int(lens[b])) if good[b] else 0
        need = max(0, want[b] - have[b]) if good[b] else 0
        asked += need
        fits = (need == 0 or asked <= room) and (
            rows == 0 or n_slots is None or offsets[-1] + rows <= n_slots)
        full |= not fits
        old = int(lens[b])
        if fits:
            for p in range(have[b], have[b] + need):
                count -= 1
                table[b, p] = stack[count]
            if good[b]:
                lens[b] = new[b]
        for t in range(old, old + rows):
            page = int(table[b, t // PAGE]) if fits else -1
            slots.append(page * PAGE + t % PAGE if 0 <= page < num_blocks else -1)
        offsets.append(offsets[-1] + rows)
    if n_slots is not None:
        slots = (slots + none)[:n_slots]
    return table, lens, stack, count, slots, offsets, full


def logprobs(logits, tokens, n_top, temperature=1.0, allowed=None):
    """logits [N, V] float64; allowed [N, V] bool.  (logprob, entropy, rank,
    top logprobs, top tokens)."""
    n, v = logits.shape
    lp, en = np.zeros(n), np.zeros(n)
    rank = np.full(n, -1, np.int32)
    top, which = np.full((n, n_top), -np.inf), np.full((n, n_top), -1, np.int32)
    for r in range(n):
        t = int(tokens[r])
        if t < 0 or t >= v:
            continue
        ok = logits[r] != -np.inf
        if allowed is not None:
            ok &= allowed[r]
        ids = np.nonzero(ok)[0]
        x = logits[r, ids]
        if len(ids) == 0:
            lp[r] = -np.inf
            continue
        z = x / temperature
        with np.errstate(invalid="ignore", over="ignore"):
            m = z.max()
            e = np.exp(z - m)
            lse = m + np.log(e.sum())
            p = e / e.sum()
            lp[r] = logits[r, t] / temperature - lse if ok[t] else (
                np.nan if np.isnan(lse) else -np.inf)
            en[r] = -np.where(p > 0, p * (z - lse), np.where(np.isnan(p), p, 0)).sum()
        # NaN above +inf, equals by index
        order = np.lexsort((ids, -np.where(np.isnan(x), np.inf, x), ~np.isnan(x)))
        if ok[t]:
            rank[r] = int(np.nonzero(ids[order] == t)[0][0])
        k = min(n_top, len(ids))
        which[r, :k] = ids[order[:k]]
        with np.errstate(invalid="ignore"):
            top[r, :k] = z[order[:k]] - lse
    return lp, en, rank, top, which
