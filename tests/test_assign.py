"""Page assignment and packed appends on the GPU, against the plain forms of
page_ref.py.  Everything here is whole numbers or stored bytes: equal."""
import numpy as np
import pytest

import cache_ref as R
import page_ref as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svp():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import spec_verify_paged_gb300 as m
    return m


class State:
    """The same batch twice: arrays for the plain form, tensors for the call."""

    def __init__(self, rng, batch, width, pages, lens=None):
        self.table = np.full((batch, width), -1, np.int32)
        self.lens = np.zeros(batch, np.int32)
        self.stack = rng.permutation(pages).astype(np.int32)
        self.count = pages
        if lens is not None:
            self.table, self.lens, self.stack, self.count, *_ = G.assign(
                self.table, self.lens, np.asarray(lens, np.int32), self.stack, pages)
        self.push()

    def push(self):
        self.g = [R.to_gpu(x) for x in (self.table, self.lens, self.stack,
                                        np.array([self.count], np.int32))]

    def go(self, svp, new, n_slots=None, num_blocks=None):
        """One call on both; the device's flags."""
        new = np.asarray(new, np.int32)
        t, n, s, c = self.g
        slots, offsets = svp.kv_assign_pages(t, n, R.to_gpu(new), s, c, n_slots=n_slots,
                                             num_blocks=num_blocks)
        (self.table, self.lens, self.stack, self.count, want, off, short) = G.assign(
            self.table, self.lens, new, self.stack, self.count, n_slots,
            2 ** 31 - 1 if num_blocks is None else num_blocks)
        flags = svp.read_device_status()
        for got, ref in ((t, self.table), (n, self.lens), (s, self.stack)):
            assert np.array_equal(got.cpu().numpy(), ref)
        assert c.tolist() == [self.count] and offsets.tolist() == off
        if n_slots is None:
            assert slots is None
        else:
            assert slots.tolist() == want
        assert bool(flags & 16) == short
        return flags


@pytest.mark.parametrize("batch,width,step,n_slots", [
    (1, 1, 16, 20), (3, 4, 20, 70), (64, 20, 40, 3000), (64, 20, 300, 20000),
    (1023, 3, 5, 6000), (1024, 3, 5, 9000), (1025, 3, 5, None), (2500, 4, 30, 80000),
])
def test_growing_and_shrinking(svp, batch, width, step, n_slots):
    rng = np.random.default_rng(batch + width)
    st = State(rng, batch, width, batch * width)
    for turn in range(6):
        new = np.clip(st.lens + rng.integers(-step, step + 1, batch), 0, 16 * width)
        if turn == 3:
            new = np.where(rng.random(batch) < 0.5, 0, new)  # half of them end
        if turn == 5:
            new[:] = 0
        assert st.go(svp, new, n_slots) == 0
    assert st.count == batch * width and (st.table == -1).all()


@pytest.mark.parametrize("n_slots", [None, 500, 30000])
def test_pages_run_out(svp, n_slots):
    """Sequences from the first that does not fit keep what they have; those
    that need no page go on.  (500 slots run out before the pages do.)"""
    rng = np.random.default_rng(7)
    st = State(rng, 200, 10, 600, rng.integers(0, 40, 200))
    for _ in range(4):
        new = np.clip(st.lens + rng.integers(-10, 40, 200), 0, 160)
        st.go(svp, new, n_slots)
    assert st.count < 30 or n_slots == 500


def test_slots_run_out(svp):
    rng = np.random.default_rng(8)
    st = State(rng, 40, 4, 160, rng.integers(0, 20, 40))
    assert st.go(svp, st.lens + 5, 199) == 16
    assert st.go(svp, st.lens + 1, 40) == 0
    assert st.go(svp, st.lens + 1, 0) == 16
    assert st.go(svp, st.lens, 0) == 0
    assert st.go(svp, np.maximum(st.lens - 3, 0), 7) == 0


def test_exactly_enough(svp):
    st = State(np.random.default_rng(9), 4, 3, 5, [1, 16, 17, 0])
    assert st.count == 1
    assert st.go(svp, [16, 16, 32, 16], 63) == 0     # the last page
    assert st.count == 0
    assert st.go(svp, [0, 17, 32, 32], 17) == 16     # one comes back, two are wanted
    assert st.lens.tolist() == [0, 17, 32, 16]


def test_bad_lengths_and_ids(svp):
    rng = np.random.default_rng(10)
    st = State(rng, 5, 3, 15, [10, 20, 30, 40, 48])
    for at, old, new in ((0, 10, -1), (1, 20, 49), (2, -7, 3), (3, 49, 0)):
        st.lens[at] = old
        st.push()
        target = st.lens.copy()
        target[at] = new
        target[4] = 20
        assert st.go(svp, target, 10) == 2
        st.lens[at] = 10
        st.table[at] = st.table[at]
        st.push()
    # ids past the cache are handed on, without slots, and flagged
    st = State(rng, 3, 3, 9, [5, 20, 0])
    assert st.go(svp, [20, 3, 40], 60, num_blocks=4) & 1


def test_inconsistent_stacks_change_nothing(svp):
    rng = np.random.default_rng(11)
    st = State(rng, 3, 3, 9, [5, 20, 0])
    for count in (-1, 10, 9):     # 9: a page would come back to a full stack
        st.count = count
        st.push()
        assert st.go(svp, [5, 3, 0], 4) == 16


def test_lengths_of_their_own_target(svp):
    """new_lens may be seq_lens itself."""
    st = State(np.random.default_rng(12), 3, 3, 9, [5, 20, 0])
    t, n, s, c = st.g
    slots, off = svp.kv_assign_pages(t, n, n, s, c, n_slots=3)
    assert slots.tolist() == [-1] * 3 and off.tolist() == [0] * 4
    assert n.tolist() == [5, 20, 0] and svp.read_device_status() == 0


def test_empty_batch_and_refusals(svp):
    import torch
    z = dict(dtype=torch.int32, device="cuda")
    t, n, c = torch.zeros((0, 3), **z), torch.zeros(0, **z), torch.ones(1, **z)
    s = torch.zeros(4, **z)
    slots, off = svp.kv_assign_pages(t, n, n, s, c, n_slots=3)
    assert slots.tolist() == [-1] * 3 and off.tolist() == [0] and c.tolist() == [1]
    t, n = torch.zeros((2, 3), **z), torch.zeros(2, **z)
    for bad in (dict(seq_lens=n[:1]), dict(new_lens=n.long()), dict(free_count=n),
                dict(block_table=t.t()), dict(n_slots=-1), dict(free_pages=s.cpu()),
                dict(slots=torch.zeros(3, **z)), dict(offsets=n)):
        args = dict(block_table=t, seq_lens=n, new_lens=n, free_pages=s, free_count=c)
        args.update(bad)
        with pytest.raises(ValueError):
            svp.kv_assign_pages(**args)


def test_captured_steps(svp):
    """A graph of an assignment, replayed: the state moves on."""
    import torch
    rng = np.random.default_rng(13)
    st = State(rng, 6, 8, 60, [3, 16, 40, 0, 1, 31])
    t, n, s, c = st.g
    target = torch.zeros(6, dtype=torch.int32, device="cuda")
    slots = torch.empty(100, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    target.copy_(n)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        svp.kv_assign_pages(t, n, target, s, c, slots=slots)
    for _ in range(5):
        new = np.clip(st.lens + rng.integers(-15, 16, 6), 0, 128).astype(np.int32)
        target.copy_(R.to_gpu(new))
        graph.replay()
        st.table, st.lens, st.stack, st.count, want, _, short = G.assign(
            st.table, st.lens, new, st.stack, st.count, 100)
        assert np.array_equal(t.cpu().numpy(), st.table) and n.tolist() == st.lens.tolist()
        assert np.array_equal(s.cpu().numpy(), st.stack) and slots.tolist() == want
    assert svp.read_device_status() == 0


# --------------------------------------------------------- packed appends

@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "fp4"])
@pytest.mark.parametrize("d,hkv,lens", [(64, 1, [1]), (128, 3, [7, 1, 20, 13]),
                                        (64, 5, [64, 3, 33]), (128, 8, [64] * 40)])
def test_packed_rows_are_stored_as_kv_append_stores_them(svp, dtype, d, hkv, lens):
    import torch
    rng = np.random.default_rng(d + hkv)
    table, total, _ = R.pages(rng, lens, spare=1)
    ks, vs = (0.0371, 0.05) if dtype in ("fp8", "fp4") else (1.0, 1.0)
    io = torch.float32 if dtype == "f32" else torch.bfloat16
    width = svp.fp4_row_bytes(d) if dtype == "fp4" else d
    ct = dict(f32=torch.float32, bf16=torch.bfloat16).get(dtype, torch.uint8)
    a, b = ([torch.zeros((total, hkv, 16, width), dtype=ct, device="cuda") for _ in "kv"]
            for _ in range(2))
    n = sum(lens)
    new = [(torch.randn((n, hkv, d), device="cuda") * 3).to(io) for _ in "kv"]
    slots, at = [], 0
    for i, m in enumerate(lens):
        pos = np.arange(m)
        slots += (table[i, pos // 16].astype(np.int64) * 16 + pos % 16).tolist()
        rows = [x[at:at + m][None].contiguous() for x in new]
        svp.kv_append(*rows, *b, R.to_gpu(table[i:i + 1]),
                      torch.tensor([m], dtype=torch.int32, device="cuda"),
                      k_scale=ks, v_scale=vs)
        at += m
    svp.kv_append(*new, *a, slots=torch.tensor(slots, device="cuda"), k_scale=ks, v_scale=vs)
    assert svp.read_device_status() == 0
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_slots_that_store_nothing(svp):
    """Negative slots store nothing, those past the cache are flagged."""
    import torch
    for dtype, width in ((torch.bfloat16, 64), (torch.uint8, 64), (torch.uint8, 36)):
        k, v = (torch.zeros((3, 2, 16, width), dtype=dtype, device="cuda") for _ in "kv")
        x = torch.ones((5, 2, 64), dtype=torch.bfloat16, device="cuda")
        slots = torch.tensor([-1, 47, 48, 2 ** 62, -2 ** 62], device="cuda")
        svp.kv_append(x, x, k, v, slots=slots)
        assert svp.read_device_status() == 1
        stored = (k != 0).flatten(3).any(-1).nonzero()
        assert stored.tolist() == [[2, 0, 15], [2, 1, 15]]
    with pytest.raises(ValueError):
        svp.kv_append(x, x, k, v, slots=slots.int())
    with pytest.raises(ValueError):
        svp.kv_append(x, x[:4], k, v, slots=slots)
    svp.kv_append(x[:0], x[:0], k, v, slots=slots[:0])


def test_slots_beyond_32_bits_of_bytes(svp):
    import torch
    nb = 2_200_000                     # 64 heads' bytes pass 2^32 in each cache
    k, v = (torch.empty((nb, 1, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    x = torch.randn((3, 1, 64), device="cuda").bfloat16()
    slots = torch.tensor([nb * 16 - 1, 0, 2_097_152 * 16 + 5], device="cuda")
    svp.kv_append(x, -x, k, v, slots=slots)
    assert svp.read_device_status() == 0
    assert torch.equal(k.view(-1, 64)[slots], x[:, 0])
    assert torch.equal(v.view(-1, 64)[slots], -x[:, 0])
