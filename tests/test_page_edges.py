"""Selected pages, page assignment and log probabilities where the other files
do not look: weights' bits, shapes that take another branch of a launcher, and
a step whose pages run out.  Tolerances as in test_page_sparse.py."""
import os
import subprocess

import numpy as np
import pytest

import cache_ref as R
import page_ref as G


@pytest.fixture(scope="module")
def svp():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import spec_verify_paged_gb300 as m
    return m


def _f64(t):
    return t.float().double().cpu().numpy()


# --------------------------------------------------- attention over a list

@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [4, 16, 24, 32])
def test_sparse_bf16_weights_keep_their_bits(svp, d, group):
    """Two keys, of weights 1 and p = exp(-q), whose values are bf16(p) and -1:
    they cancel up to the bits of p that bf16 does not hold.  A weight in two
    bf16 terms is off by 2^-8 of 2^-8 of itself, its exponent by the 3 roundings
    of at most 2 log2(e) (2^-24 each), the sums and the division by 2^-21."""
    rng = np.random.default_rng(group + d)
    q = np.zeros((1, 1, group, d))
    q[..., 0] = R.bf16(rng.uniform(0.2, 2.0, group))
    k = np.zeros((1, 1, 16, d))
    k[0, 0, 1, 0] = -1.0
    v = np.zeros((1, 1, 16, d))
    v[0, 0, 0] = R.bf16(np.exp(-np.resize(q[0, 0, :, 0], d)))
    v[0, 0, 1] = -1.0
    one = np.zeros((1, 1, 1), np.int32)
    out, lse = svp.paged_sparse_attention(
        *(R.to_gpu(x.astype(np.float32), "bf16") for x in (q, k, v)),
        R.to_gpu(one[0]), R.to_gpu(np.array([2], np.int32)), R.to_gpu(one), scale=1.0)
    want, wlse, _, _ = G.sparse_attention(q, k, v, 1.0, [2], one[0], one)
    assert svp.read_device_status() == 0
    tol = 2.0 ** -16 + 3 * 3 * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -8 * np.abs(want)
    assert (np.abs(_f64(out) - want) <= tol).all()
    assert np.abs(_f64(lse) - wlse).max() <= 2.0 ** -20


SPLITS = r"""
#include <cstdio>
#include "svp.h"
#include "svp_internal.h"
int main() {
  long long units;
  int n_select, split_pages, sms, per_sm, f32, fit;
  while (std::scanf("%lld %d %d %d %d %d %d", &units, &n_select, &split_pages, &sms,
                    &per_sm, &f32, &fit) == 7) {
    int asked = 0;
    const int n = svp::sparse_splits(units, n_select, split_pages, sms, per_sm, f32 != 0,
                                     [&] { ++asked; return fit != 0; });
    std::printf("%d %d\n", n, asked);
  }
}
"""


@pytest.fixture(scope="module")
def splits(tmp_path_factory):
    """The launcher's rule, as host code: {(units, list, split_pages, SMs, CTAs an
    SM holds, fp32, sixteen fit): (CTAs to a unit, asked whether they fit)}."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = tmp_path_factory.mktemp("splits")
    (path / "splits.cpp").write_text(SPLITS)
    exe = str(path / "splits")
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(cuda, "include"), "-I",
                    os.path.join(root, "include"), "-I",
                    os.path.join(root, "spec_verify_paged_gb300", "csrc"),
                    str(path / "splits.cpp"), "-o", exe], check=True)

    def check(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, check=True)
        got = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
        assert dict(zip(cases, got)) == cases and len(got) == len(cases)

    return check


def test_clusters_of_sixteen_where_the_device_has_them(splits):
    """Sixteen CTAs to a list only where the device says that it can place them,
    eight where it cannot, and no question where sixteen are not wanted."""
    splits({(1, 2048, 0, 152, 2, 0, 1): (16, 1), (1, 2048, 0, 152, 2, 0, 0): (8, 1),
            (1, 2048, 0, 152, 1, 1, 1): (16, 1), (1, 2048, 0, 152, 1, 1, 0): (8, 1),
            # eight entries to a CTA: sixteen CTAs from 16 * 8 = 128 entries on
            (1, 255, 0, 152, 2, 0, 1): (16, 1), (1, 128, 0, 152, 2, 0, 1): (16, 1),
            (1, 127, 0, 152, 2, 0, 1): (8, 0), (64, 256, 0, 152, 2, 0, 1): (4, 0),
            (1, 16, 1, 152, 2, 0, 1): (16, 1), (1, 16, 1, 152, 2, 0, 0): (8, 1),
            (256, 128, 0, 152, 2, 0, 1): (1, 0), (256, 128, 16, 152, 2, 0, 1): (8, 0),
            (1, 1, 0, 152, 2, 0, 1): (1, 0), (1, 2048, 0, 15, 2, 0, 1): (8, 0),
            (1 << 40, 1 << 26, 1 << 26, 152, 2, 0, 1): (1, 0)})


def test_lists_are_split_into_ctas_that_find_room(splits):
    """As many CTAs as the SMs hold, one or two to an SM."""
    splits({(units, 128, 0, 152, per, f32, 1): (n, 0)
            for per, f32 in ((2, 0), (2, 1), (1, 1))
            for units, n in ((20 * per, 4), (32 * per, 4), (38 * per, 4), (39 * per, 2),
                             (76 * per, 2), (77 * per, 1), (152 * per, 1))})


# ------------------------------------------- a step whose pages run out

def _documented_step():
    """The step over selected pages as it is published: what stands before it, and
    the step."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        blocks = f.read().split("```python\n")[1:]
    block, = (x for x in (b.split("```")[0] for b in blocks) if "kv_assign_pages(" in x)
    at = block.index("\n") + 1
    assert block[:at].startswith("bounds = ")
    return block[:at], block[at:]


class Short:
    """Six sequences whose five new rows want four new pages, of which there is
    one: the first gets it, the fourth and the fifth need none."""
    B, q_len, Hkv, D, num_blocks, vocab = 6, 5, 2, 64, 24, 40

    def __init__(self, device):
        import torch
        rng = np.random.default_rng(31)
        lens = np.array([60, 16, 31, 200, 3, 0], np.int32)
        self.table, _, _ = R.pages(rng, lens, width=16)
        used = self.table[self.table >= 0]
        stack = np.setdiff1d(np.arange(self.num_blocks), used).astype(np.int32)
        self.lens, self.count = lens, 1
        self.stack = np.concatenate([stack[:1], np.zeros(self.num_blocks - 1, np.int32)])
        g = torch.Generator().manual_seed(3)

        def rand(*shape):
            return torch.randn(shape, generator=g).to(device)

        def ints(x):
            return torch.from_numpy(np.array(x, np.int32)).to(device)

        n = (self.B * self.q_len, self.Hkv, self.D)
        cache = (self.num_blocks, self.Hkv, 16, self.D)
        target = rand(self.B, self.q_len, self.vocab)
        draft = target[:, :-1] + 0.3 * rand(self.B, self.q_len - 1, self.vocab)
        self.names = dict(
            torch=torch, B=self.B, q_len=self.q_len, Hkv=self.Hkv, D=self.D,
            num_blocks=self.num_blocks, block_table=ints(self.table), seq_lens=ints(lens),
            free_pages=ints(self.stack), free_count=ints([1]),
            k_new=rand(*n).bfloat16(), v_new=rand(*n).bfloat16(),
            k_cache=rand(*cache).bfloat16(), v_cache=rand(*cache).bfloat16(),
            q=rand(self.B, self.q_len, 2 * self.Hkv, self.D).bfloat16(),
            target_logits=target, draft_logits=draft,
            draft_tokens=draft.argmax(-1).int(),
            uniforms=torch.rand((self.B, self.q_len), generator=g).to(device))

    def check(self):
        """After a step: the state of the plain form, in which a sequence that
        got its pages keeps what it accepted and the others all they had."""
        x = self.names
        old, want = self.lens, self.lens + self.q_len
        before = [self.table.copy(), old.copy()]
        self.table, self.lens, self.stack, self.count, *_ = G.assign(
            self.table, old, want, self.stack, self.count, self.B * self.q_len)
        served = self.lens == want
        accepted = x["n_accepted"].cpu().numpy()
        self.table, self.lens, self.stack, self.count, *_ = G.assign(
            self.table, self.lens, np.where(served, old + 1 + accepted, old), self.stack,
            self.count)
        assert np.array_equal(x["seq_lens"].cpu().numpy(), self.lens)
        assert np.array_equal(x["block_table"].cpu().numpy(), self.table)
        assert x["free_count"].tolist() == [self.count]
        assert np.array_equal(x["free_pages"].cpu().numpy(), self.stack)
        assert np.array_equal(self.table[~served], before[0][~served])
        assert np.array_equal(self.lens[~served], before[1][~served])
        tokens = x["tokens"].cpu().numpy()
        assert (tokens[~served] == -1).all() and (tokens[served, 0] >= 0).all()
        return served


def test_the_documented_step_keeps_rows_when_pages_run_out():
    """Its arithmetic on the host, with the plain form of the assignment."""
    import types

    import torch
    short = Short("cpu")
    x = short.names

    def assign(table, lens, new, free, count, n_slots=None):
        t, n, s, c, slots, off, _ = G.assign(
            *(a.numpy() for a in (table, lens, new, free)), int(count), n_slots)
        for to, a in ((table, t), (lens, n), (free, s)):
            to.copy_(torch.from_numpy(a))
        count.fill_(c)
        return (None if n_slots is None else torch.tensor(slots)), torch.tensor(off)

    def accept(*_):
        n = (torch.arange(short.B) + turn).int() % short.q_len
        return torch.zeros((short.B, short.q_len), dtype=torch.int32), n

    def five(*_, **__):
        return (None,) * 5

    def two(*_, **__):
        return None, None

    x["svp"] = types.SimpleNamespace(
        kv_assign_pages=assign, spec_accept=accept, token_logprobs=five,
        paged_sparse_attention=two, kv_append=two, kv_page_bounds=two,
        paged_page_scores=two, paged_select_pages=two)
    first, step = _documented_step()
    exec(first.replace('"cuda"', '"cpu"'), x)
    for turn in range(6):
        exec(step, x)
        served = short.check()
        if turn == 0:
            assert served.tolist() == [True, False, False, True, True, False]


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_the_documented_step_when_pages_run_out(svp, captured):
    """The step itself, as calls and as a graph: committed rows stay, and rows
    that no page was found for are stored nowhere."""
    import torch
    short = Short("cuda")
    x = short.names
    x["svp"] = svp
    first, step = _documented_step()
    exec(first, x)
    step = compile(step, "step", "exec")
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            exec(step, x)
    for _ in range(4):
        k, old, table = (x[n].clone() for n in ("k_cache", "seq_lens", "block_table"))
        graph.replay() if captured else exec(step, x)
        served = short.check()
        # no page for some, and nothing but an empty sequence's length besides
        assert svp.read_device_status() & ~2 == (0 if served.all() else 16)
        kc = x["k_cache"]
        for b, n in enumerate(old.tolist()):  # the rows there were
            for j in range(-(-n // 16)):
                r = min(16, n - 16 * j)
                assert torch.equal(kc[table[b, j], :, :r], k[table[b, j], :, :r])
        rank = x["rank"].cpu().numpy()
        assert (rank[~served] == -1).all() and (rank[served, 0] >= 0).all()


# ----------------------------------------- who is served when things run out

#          lengths and targets          free  slots  served
SHORTAGES = [
    # the second needs two pages of one; behind it only those that need none:
    # within a page, shorter (whose page came back before), the same, but not
    # the last, which needs one
    ([16, 16, 20, 40, 5, 16], [20, 60, 32, 20, 5, 17], 1, None, [0, 2, 3, 4]),
    # the second's four positions do not fit; behind it only those without any
    ([3, 3, 3, 40, 5, 3], [5, 7, 4, 20, 5, 4], 0, 5, [0, 3, 4]),
    # entries run out before pages do
    ([0, 0, 0, 0, 20, 0], [16, 16, 1, 0, 19, 0], 4, 20, [0, 3, 4, 5]),
]


def _shortage(lens, new, free, slots):
    rng = np.random.default_rng(5)
    table, total, _ = R.pages(rng, np.array(lens, np.int32), width=4)
    stack = np.full(40, -7, np.int32)
    stack[:free] = total + np.arange(free)
    return table, np.array(lens, np.int32), np.array(new, np.int32), stack, free, slots


@pytest.mark.parametrize("lens,new,free,slots,served", SHORTAGES)
def test_who_is_served_plain(lens, new, free, slots, served):
    table, old, new, stack, count, slots = _shortage(lens, new, free, slots)
    t, n, *_, short = G.assign(table, old, new, stack, count, slots)
    assert short and np.nonzero(n == new)[0].tolist() == served
    rest = n != new
    assert np.array_equal(t[rest], table[rest]) and np.array_equal(n[rest], old[rest])


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new,free,slots,served", SHORTAGES)
def test_who_is_served(svp, lens, new, free, slots, served):
    table, old, new, stack, count, slots = _shortage(lens, new, free, slots)
    t, n, s = (R.to_gpu(x) for x in (table, old, stack))
    c = R.to_gpu(np.array([count], np.int32))
    svp.kv_assign_pages(t, n, R.to_gpu(new), s, c, n_slots=slots)
    assert svp.read_device_status() == 16
    got = n.cpu().numpy()
    assert np.nonzero(got == new)[0].tolist() == served
    rest = got != new
    assert np.array_equal(t.cpu().numpy()[rest], table[rest])
    assert np.array_equal(got[rest], old[rest])


# ------------------------------------ shapes that take another branch

def _sms():
    import torch
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,hkv", [
    ("fp8", 128, 3), ("fp8", 128, 4), ("fp8", 64, 7), ("fp8", 64, 2), ("fp4", 128, 8),
    ("fp4", 128, 1), ("fp4", 64, 9), ("fp4", 64, 5), ("bf16", 64, 3), ("bf16", 64, 2),
])
@pytest.mark.parametrize("n_new", [None, 40])
def test_bounds_several_heads_to_a_warp(svp, dtype, d, hkv, n_new):
    """From 256 (page, head) pairs to an SM on a warp takes several heads of a
    page, also where that leaves fewer for the last one.  What counts are the
    pages a call may touch: the table's width, or four of each sequence."""
    rng = np.random.default_rng(d + hkv)
    pairs = 256 * _sms()
    batch = 7 if n_new is None else pairs // (4 * hkv) + 7
    width = pairs // (7 * hkv) + 1 if n_new is None else 5
    lens = np.zeros(batch, np.int32)
    lens[:7] = [0, 1, 16, 17, 64, 33, 300 if n_new is None else 48]
    table, total, _ = R.pages(rng, lens, spare=3, width=width)
    scale = {"fp8": 2.0 ** -5, "fp4": 0.0371}.get(dtype, 1.0)
    k = R.make_cache(rng, dtype, total, hkv, d, scale, lens, table)
    old = rng.integers(-3, 4, (total, hkv, 2, d)).astype(np.float64)
    b = R.to_gpu(old.astype(np.float32), "bf16")
    svp.kv_page_bounds(R.to_gpu(k, "bf16" if dtype == "bf16" else None),
                       R.to_gpu(table), R.to_gpu(lens), b, n_new)
    assert svp.read_device_status() == 0
    want = G.bounds(R.values(k, dtype, d), lens, table, n_new or 10 ** 6, old)
    assert np.array_equal(_f64(b), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group,ql", [(2, 1), (8, 4), (8, 5)])
def test_scores_short_parts(svp, dtype, group, ql):
    """More (sequence, head) pairs than CTAs at once and more than 48 tiles of
    16 pages: the pages are cut into parts of 20 tiles, of 32 with 33 rows and
    more.  Tolerance as in test_page_sparse.py."""
    rng = np.random.default_rng(group + ql)
    d, hkv = 64, 8
    batch, width = 4 * _sms() // hkv + 1, 16 * 49 + 3
    lens = np.full(batch, ql, np.int32)
    lens[[0, 2, batch - 1]] = [16 * width, 16 * 600 + 1, 16 * 321]
    table, total, _ = R.pages(rng, lens, width=width)
    mid = rng.standard_normal((total, hkv, 1, d))
    bnd = R.bf16(np.concatenate([mid - 1.5, mid + 1.5], 2))
    q = rng.standard_normal((batch, ql, hkv * group, d))
    q = q.astype(np.float32).astype(np.float64) if dtype == "f32" else R.bf16(q)
    got = svp.paged_page_scores(
        R.to_gpu(q.astype(np.float32), None if dtype == "f32" else "bf16"),
        R.to_gpu(bnd.astype(np.float32), "bf16"), R.to_gpu(table), R.to_gpu(lens),
        scale=0.125)
    assert svp.read_device_status() == 0
    want, mag = G.scores(q, bnd, lens, table, 0.125)
    got = _f64(got)
    live = np.isfinite(want)
    assert np.array_equal(live, np.isfinite(got)) and (got[~live] == -np.inf).all()
    n = 2 * d * (3 if dtype == "f32" else 1) + 4
    assert (np.abs(got[live] - want[live]) <= n * 2.0 ** -23 * mag[live]).all()


@pytest.mark.gpu
def test_assign_without_slots_by_eight_ctas(svp):
    """Up to 1024 sequences and more than 4096 table entries, without slots."""
    from test_assign import State
    rng = np.random.default_rng(51)
    for batch, width in ((700, 8), (1024, 5), (3, 2000)):
        st = State(rng, batch, width, batch * width - batch // 2)
        for turn in range(4):
            new = rng.integers(0, 16 * width + 1, batch)
            assert st.go(svp, new) in (0, 16)
        assert st.go(svp, np.zeros(batch)) == 0
        assert st.count == batch * width - batch // 2


# --------------------------------------------------- the device's flags

@pytest.mark.gpu
def test_status_read_is_one_round_trip(svp):
    """Reading the flags waits for the GPU once, not once or twice for each
    source file that has some: at most five times what one number read back
    takes (12 pairs of copies and waits take sixteen)."""
    import time

    import torch
    x = torch.zeros(1, device="cuda")

    def best(f):
        t = []
        for _ in range(200):
            t0 = time.perf_counter()
            f()
            t.append(time.perf_counter() - t0)
        return min(t)

    svp.read_device_status()
    one, status = best(x.item), best(svp.read_device_status)
    print(f"{1e6 * one:.1f} us, {1e6 * status:.1f} us")
    assert status <= 5 * one


@pytest.mark.gpu
def test_status_of_several_files_and_threads(svp):
    """Flags of several files arrive together and once, and threads that read at
    the same time get every flag between them."""
    import threading

    import torch
    z = dict(dtype=torch.int32, device="cuda")
    table, lens = torch.full((1, 2), 99, **z), torch.tensor([40], **z)

    def raise_all():
        svp.paged_select_pages(torch.zeros((1, 1, 2), device="cuda"), lens, 1)      # 2
        svp.kv_assign_pages(table, torch.tensor([0], **z), torch.tensor([16], **z),
                            torch.zeros(1, **z), torch.zeros(1, **z))               # 16
        svp.token_logprobs(torch.zeros((1, 8), device="cuda"), torch.tensor([9], **z))  # 4
        svp.kv_page_bounds(torch.zeros((4, 1, 16, 64), device="cuda"), table,
                           torch.tensor([5], **z),
                           torch.zeros((4, 1, 2, 64), dtype=torch.bfloat16,
                                       device="cuda"))                              # 1
    svp.read_device_status()
    raise_all()
    assert svp.read_device_status() == 1 | 2 | 4 | 16
    assert svp.read_device_status() == 0
    for _ in range(20):
        raise_all()
        torch.cuda.synchronize()
        got = []

        def read():
            with torch.cuda.stream(torch.cuda.Stream()):
                got.append(svp.read_device_status())

        threads = [threading.Thread(target=read) for _ in range(6)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert np.bitwise_or.reduce(got) == 1 | 2 | 4 | 16
        assert svp.read_device_status() == 0
