"""Host-side checks and planning of the attention, score and build layers (no
GPU)."""
import ctypes

import pytest

P = ctypes.c_void_p(0x1000)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from spec_verify_paged_gb300 import binding, build
    build.build()
    return binding.load_library()


def _dims(**kw):
    from spec_verify_paged_gb300.binding import SvpDims
    d = SvpDims()
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128,
                block_size=16, max_blocks_per_seq=4, num_blocks=8, dtype=3,
                k_scale=1.0, v_scale=1.0)
    base.update(kw)
    for k, v in base.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("dtype", [0, 1, 2, 3])
@pytest.mark.parametrize("off", [1, 4, 8])
def test_workspace_alignment(lib, dtype, off):
    """Partials move as 16-byte vectors and bulk copies: a workspace that is
    not 16-byte aligned is refused before anything is launched."""
    d = _dims(dtype=dtype, workspace=P.value + off, workspace_bytes=1 << 30)
    assert lib.paged_decode_attention(ctypes.byref(d), P, P, P, P, P, 1, 0, 0, 0.1,
                                      P, P, None) == -1
    assert lib.paged_tree_attention(ctypes.byref(d), P, P, P, P, P, 2, P, 0.1, P, P,
                                    None) == -1
    assert lib.svp_last_launch_count() == 0


@pytest.mark.parametrize("dtype", [1, 3])
@pytest.mark.parametrize("n_sink", [2 ** 31 - 16, 2 ** 31 - 15, 2 ** 31 - 1])
def test_any_number_of_sinks_plans_the_whole_table(lib, dtype, n_sink):
    """Sinks beyond any length: the visible pages are the table's, as without
    a window."""
    d = _dims(dtype=dtype, batch=8, max_blocks_per_seq=4096, num_blocks=4096)
    all_pages = lib.paged_decode_workspace_size(ctypes.byref(d), 1, 0, 0)
    assert all_pages > 256
    for window in (1, 16, 2 ** 31 - 1):
        assert lib.paged_decode_workspace_size(ctypes.byref(d), 1, n_sink,
                                               window) == all_pages
