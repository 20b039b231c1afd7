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


# ------------------------------------------- the marshalling module's build

@pytest.fixture
def calls_build(lib, tmp_path, monkeypatch):
    """The build layer with a stand-in for the built module, up to date."""
    from spec_verify_paged_gb300 import build
    monkeypatch.setattr(build, "CALLS_LIB", str(tmp_path / "svp_calls.so"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    made = []

    def compile_calls():
        made.append("compiled")
        return "calls.o"

    def link(obj):
        (tmp_path / "svp_calls.so").write_bytes(b"")
    monkeypatch.setattr(build, "_compile_calls", compile_calls)
    monkeypatch.setattr(build, "_link_calls", link)
    build.build()
    assert made == ["compiled"]
    build.build()
    assert made == ["compiled"]     # up to date
    return build, made


@pytest.mark.parametrize("change", ["torch", "python", "place"])
def test_another_torch_or_python_rebuilds_the_module(calls_build, monkeypatch, change):
    build, made = calls_build
    import importlib.metadata
    import importlib.util
    import sysconfig
    if change == "torch":
        monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0.1")
    elif change == "python":
        old = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var",
                            lambda k: "other" if k == "SOABI" else old(k))
    else:
        class Spec:
            origin = "/somewhere/else/torch/__init__.py"
        monkeypatch.setattr(importlib.util, "find_spec", lambda name: Spec)
    build.build()
    assert made == ["compiled"] * 2
    build.build()
    assert made == ["compiled"] * 2


def test_a_module_that_does_not_build_is_named(calls_build, monkeypatch):
    """The library is in place all the same, and the error says what is not."""
    import os
    build, _ = calls_build

    def fail():
        raise RuntimeError("no Python.h")
    monkeypatch.setattr(build, "_compile_calls", fail)
    os.remove(build.CALLS_LIB)
    with pytest.raises(RuntimeError, match="svp_calls.*libsvp.so is in place.*no Python.h"):
        build.build()
    assert os.path.exists(build.LIB)


def test_a_module_of_another_torch_is_not_loaded(lib, monkeypatch):
    torch = pytest.importorskip("torch")
    from spec_verify_paged_gb300 import binding
    monkeypatch.setattr(binding, "_calls", None)
    assert binding._load_calls() is not None
    monkeypatch.setattr(binding, "_calls", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="0.0.1"):
        binding._load_calls()
    assert binding._calls is None
