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
  int n_select, split_pages, sms, f32, fit;
  while (std::scanf("%lld %d %d %d %d %d", &units, &n_select, &split_pages, &sms, &f32,
                    &fit) == 6) {
    int asked = 0;
    const int n = svp::sparse_splits(units, n_select, split_pages, sms, f32 != 0,
                                     [&] { ++asked; return fit != 0; });
    std::printf("%d %d\n", n, asked);
  }
}
"""


def test_clusters_of_sixteen_where_the_device_has_them(tmp_path):
    """The launcher's rule, as host code: sixteen CTAs to a list only where the
    device says that it can place them, eight where it cannot, and no question
    where sixteen are not wanted."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    (tmp_path / "splits.cpp").write_text(SPLITS)
    exe = str(tmp_path / "splits")
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(cuda, "include"), "-I",
                    os.path.join(root, "include"), "-I",
                    os.path.join(root, "spec_verify_paged_gb300", "csrc"),
                    str(tmp_path / "splits.cpp"), "-o", exe], check=True)
    #  units, list, split_pages, SMs, fp32, sixteen fit -> CTAs to a unit, asked
    cases = {(1, 2048, 0, 152, 0, 1): (16, 1), (1, 2048, 0, 152, 0, 0): (8, 1),
             (1, 2048, 0, 152, 1, 1): (16, 1), (1, 2048, 0, 152, 1, 0): (8, 1),
             # eight entries to a CTA: sixteen CTAs from 16 * 8 = 128 entries on
             (1, 255, 0, 152, 0, 1): (16, 1), (1, 128, 0, 152, 0, 1): (16, 1),
             (1, 127, 0, 152, 0, 1): (8, 0), (64, 256, 0, 152, 0, 1): (4, 0),
             (1, 16, 1, 152, 0, 1): (16, 1), (1, 16, 1, 152, 0, 0): (8, 1),
             (256, 128, 0, 152, 0, 1): (1, 0), (256, 128, 16, 152, 0, 1): (8, 0),
             (1, 1, 0, 152, 0, 1): (1, 0), (1, 2048, 0, 15, 0, 1): (8, 0),
             (1 << 40, 1 << 26, 1 << 26, 152, 0, 1): (1, 0)}
    text = "\n".join(" ".join(map(str, c)) for c in cases)
    r = subprocess.run([exe], input=text, capture_output=True, text=True, check=True)
    got = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    assert got == list(cases.values())
