"""Plain 64-bit forms of the 4-bit cache format, attention over any cache,
accumulated attention weight and eviction (numpy, loops over sequences and
heads), and seeded inputs for their tests.  A bf16 array is carried as the
float64 values it holds."""
import numpy as np

PAGE = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16(x):
    """Nearest bfloat16, ties to even, as float64 (finite input)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    u = (u + ((u >> 16) & 1) + 0x7FFF) & np.uint32(0xFFFF0000)
    return u.view(np.float32).astype(np.float64)


def e4m3_table():
    out = np.empty(256)
    for u in range(256):
        e, m = (u >> 3) & 15, u & 7
        v = (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        out[u] = np.nan if (u & 127) == 127 else (-v if u & 128 else v)
    return out


E4M3 = e4m3_table()


def e4m3_code(x):
    """Code of the nearest finite E4M3 value (ties: even code), x >= 0."""
    grid = E4M3[:127]
    x = np.minimum(x, 448.0)
    hi = np.clip(np.searchsorted(grid, x), 1, 126)
    lo = hi - 1
    d = (x - grid[lo]) - (grid[hi] - x)
    return np.where((d > 0) | ((d == 0) & (hi % 2 == 0)), hi, lo)


def quantise(x, scale_factor):
    """Values [..., D] -> 4-bit rows [..., D/2 + D/16] uint8, by the
    definition: y = x / scale_factor, scale = E4M3(max|y| / 6) in [2^-9, 448],
    code = E2M1(y / scale), the quotients rounded to fp32."""
    f32 = np.float32
    y = (x.astype(f32) / f32(scale_factor)).astype(f32)
    blocks = y.reshape(y.shape[:-1] + (-1, 16))
    top = np.abs(blocks).max(-1)
    sc = np.maximum(e4m3_code((top / f32(6)).astype(np.float64)), 1)
    r = (np.abs(blocks) / E4M3[sc].astype(f32)[..., None]).astype(np.float64)
    code = np.zeros(r.shape, np.uint8)
    for i in range(1, 8):
        mid = (E2M1[i - 1] + E2M1[i]) / 2
        code[(r > mid) | ((r == mid) & (i % 2 == 0))] = i
    code |= (blocks < 0).astype(np.uint8) << 3
    code = code.reshape(y.shape)
    byte = code[..., 0::2] | (code[..., 1::2] << 4)
    return np.concatenate([byte, sc.astype(np.uint8)], -1)


def values(rows, dtype, d, scale_factor=1.0):
    """Stored rows -> float64 values.  fp4: uint8 rows; fp8: uint8 codes."""
    if dtype == "fp4":
        byte = rows[..., :d // 2]
        code = np.stack([byte & 15, byte >> 4], -1).reshape(rows.shape[:-1] + (d,))
        v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
        return v * np.repeat(E4M3[rows[..., d // 2:]], 16, -1) * scale_factor
    if dtype == "fp8":
        return E4M3[rows] * scale_factor
    return rows.astype(np.float64)


def visible(L, q_len, i, n_sink=0, window=0, tree=None):
    """Boolean [L]: the keys query i of a sequence of length L sees."""
    j = np.arange(L)
    base, t = L - q_len, L - q_len + i
    ok = j <= t
    if tree is not None:
        bit = (int(tree[i]) >> np.clip(j - base, 0, 31)) & 1
        ok &= (j < base) | (bit == 1)
    if window:
        ok &= (j < n_sink) | (j > t - window)
    return ok


def logical(cache, table_row, h, L):
    """Rows 0..L-1 of head h of one sequence."""
    ids = table_row[:-(-L // PAGE)]
    return cache[ids, h].reshape((-1,) + cache.shape[3:])[:L]


def attention(q, k, v, scale, lens, table, n_sink=0, window=0, tree=None):
    """out, lse of the definition; q, k, v float64 values (k, v paged).  Also
    the spread sum|q||k| * |scale| (largest over the visible keys) that the
    error of a product sum is relative to, and max|v| per row."""
    B, ql, hq, d = q.shape
    per = hq // k.shape[1]
    out, lse = np.zeros((B, ql, hq, d)), np.zeros((B, ql, hq))
    mag, vmax = np.zeros((B, ql, hq)), np.zeros((B, ql, hq))
    for b in range(B):
        L = int(lens[b])
        for h in range(hq):
            kk = logical(k, table[b], h // per, L)
            vv = logical(v, table[b], h // per, L)
            for i in range(ql):
                ok = visible(L, ql, i, n_sink, window,
                             None if tree is None else tree[b])
                x = kk[ok] @ q[b, i, h] * scale
                m = x.max()
                p = np.exp(x - m)
                out[b, i, h] = p @ vv[ok] / p.sum()
                lse[b, i, h] = m + np.log(p.sum())
                mag[b, i, h] = (np.abs(kk[ok]) @ np.abs(q[b, i, h])).max() * abs(scale)
                vmax[b, i, h] = np.abs(vv[ok]).max()
    return out, lse, mag, vmax


def score_update(q, k, lse, scale, lens, table, scores, n_fresh, n_sink=0,
                 window=0, tree=None):
    """Scores after the update (a copy), and the weights added."""
    new, added = scores.astype(np.float64).copy(), np.zeros(scores.shape)
    B, ql, hq, d = q.shape
    per = hq // k.shape[1]
    for b in range(B):
        L = int(lens[b])
        for g in range(k.shape[1]):
            w = np.zeros(L)
            for i in range(ql):
                ok = visible(L, ql, i, n_sink, window,
                             None if tree is None else tree[b])
                for h in range(g * per, (g + 1) * per):
                    if lse[b, i, h] == -np.inf:
                        continue
                    x = logical(k, table[b], g, L)[ok] @ q[b, i, h] * scale
                    w[ok] += np.exp(x - lse[b, i, h])
            for j in range(L):
                at = table[b, j // PAGE], g, j % PAGE
                if j >= L - n_fresh:
                    new[at] = 0.0
                new[at] += w[j]
                added[at] = w[j]
    return new, added


def evict(scores, lens, table, budget, n_sink, n_recent, hkv):
    """kept [B, Hkv, budget] (-1 padded) and new lengths."""
    B = len(lens)
    kept = np.full((B, hkv, budget), -1, np.int32)
    for b in range(B):
        L = int(lens[b])
        for h in range(hkv):
            if L <= budget:
                keep = np.arange(L)
            else:
                s = logical(scores[..., None], table[b], h, L)[:, 0].astype(np.float64)
                s = np.where(np.isnan(s), -np.inf, s)
                mid = np.arange(n_sink, L - n_recent)
                best = np.argsort(-s[mid], kind="stable")[:budget - n_sink - n_recent]
                keep = np.sort(np.concatenate([np.arange(n_sink), mid[best],
                                               np.arange(L - n_recent, L)]))
            kept[b, h, :len(keep)] = keep
    return kept, np.minimum(lens, budget).astype(np.int32)


# ------------------------------------------------------------------ inputs

def pages(rng, lens, spare=0, width=None):
    """Block table over shuffled pages, -1 where there is none, and the ids
    left over."""
    n = -(-np.asarray(lens) // PAGE)
    total = int(n.sum()) + spare
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), max(1, width or int(n.max()))), -1, np.int32)
    at = 0
    for b, c in enumerate(n):
        table[b, :c] = perm[at:at + c]
        at += c
    return table, total, perm[at:]


def make_cache(rng, dtype, total, hkv, d, scale=1.0, lens=None, table=None):
    """Random rows as stored; with lens, every row no sequence holds is
    poisoned (NaN, for fp4 NaN scales)."""
    x = rng.standard_normal((total, hkv, PAGE, d))
    if dtype == "fp4":
        rows = quantise(x, scale)
        bad = np.uint8(0xFF)
    elif dtype == "fp8":
        sign = np.where(x < 0, 128, 0)
        rows = (e4m3_code(np.abs(x) / scale) + sign).astype(np.uint8)
        bad = np.uint8(0x7F)
    else:
        rows = (bf16(x) if dtype == "bf16" else x).astype(np.float32)
        bad = np.float32(np.nan)
    if lens is not None:
        free = np.ones((total, PAGE), bool)
        for b, L in enumerate(lens):
            for j in range(int(L)):
                free[table[b, j // PAGE], j % PAGE] = False
        rows.transpose(0, 2, 1, 3)[free] = bad
    return rows


def to_gpu(a, dtype=None):
    """numpy -> GPU tensor; dtype "bf16": float values to bfloat16."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    if dtype == "bf16":
        return t.to(torch.bfloat16).cuda()
    return t.cuda()


def binary_tree(q_len):
    bits = [1]
    for c in range(1, q_len):
        bits.append(bits[(c - 1) // 2] | (1 << c))
    return np.array(bits, np.int32)
