"""The build of the C library does not hang on torch (no GPU needed): a machine with the
CUDA toolkit alone gets the library, and a binding compiled for another torch is not
taken for this one's."""
import os
import shutil
import subprocess
import sys

import pytest

from serving_gdn_decode_gb300 import build as b


@pytest.fixture
def small(tmp_path, monkeypatch):
    """The build in a folder of its own, with one short source."""
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("needs nvcc")
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int gdn_one() { return 1; }\n')
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libgdn_gb300.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_paged_binding.so"))
    monkeypatch.setattr(b, "HERE", str(tmp_path))
    monkeypatch.setattr(b, "_sources", lambda: [str(src)])
    return tmp_path


def no_torch(monkeypatch):
    import importlib.util
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_the_library_is_built_without_torch(small, monkeypatch):
    no_torch(monkeypatch)
    assert not b.up_to_date()
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not os.path.exists(b.BINDING) and b.up_to_date()


def test_the_library_is_built_where_the_binding_does_not_compile(small, monkeypatch):
    broken = small / "broken.cpp"
    broken.write_text("#error no headers here\n")
    monkeypatch.setattr(b, "BINDING_SRC", str(broken))
    with pytest.raises(RuntimeError, match="no headers here"):  # loudly: its operators would be missing
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING) and not b.up_to_date()


def test_a_binding_of_another_torch_is_stale(small, monkeypatch):
    import importlib.metadata
    plain = small / "plain.cpp"
    plain.write_text("int gdn_plain() { return 2; }\n")
    monkeypatch.setattr(b, "BINDING_SRC", str(plain))
    b.build()
    assert os.path.exists(b.BINDING) and b.up_to_date()
    lib_time = os.path.getmtime(b.LIB)
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.1")
    assert not b.up_to_date()
    before = os.stat(b.BINDING).st_ino
    b.build()
    assert b.up_to_date() and os.stat(b.BINDING).st_ino != before and os.path.getmtime(b.LIB) == lib_time


def test_a_missing_binding_is_an_error_of_its_calls_only():
    """Without it everything else imports as ever, by name and by star, and the calls that need it say what is missing."""
    code = ("import sys\n"
            "sys.modules['serving_gdn_decode_gb300._paged_binding'] = None\n"
            "from serving_gdn_decode_gb300 import *\n"
            "assert pack_params(64, 64, 1, 1, 1, 1) is not None and gdn_forward and GdnError\n"
            "for call in (lambda: gdn_rope(*[None] * 6), lambda: gdn_rope_store(*[None] * 9), lambda: gdn_kv_plan(*[None] * 14),\n"
            "             lambda: gdn_attn_paged(*[None] * 8), lambda: gdn_attn_workspace_size(None, None, 1)):\n"
            "    try:\n"
            "        call()\n"
            "    except RuntimeError as e:\n"
            "        assert 'serving_gdn_decode_gb300.build' in str(e), e\n"
            "    else:\n"
            "        raise AssertionError('no error')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=b.ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
