"""The binding without its native part: everything loads, and every call goes the
general path."""
import os
import sysconfig

import pytest
import torch

from protein_folding_triangle_gb300 import build as B
from protein_folding_triangle_gb300 import triattn as T


@pytest.fixture()
def fresh(monkeypatch):
    B.build()
    monkeypatch.setattr(T, "_LIB", None)
    monkeypatch.setattr(T, "_HOST", None)
    return monkeypatch


def test_missing(fresh, tmp_path):
    fresh.setattr(B, "host_path", lambda: str(tmp_path / "none.so"))
    with pytest.warns(RuntimeWarning, match="native part"):
        lib = T.load()
    assert lib.triattn_status_string(0) and T.load() is lib
    host = T._host()
    assert host.qk_norm_fwd(1, 2, 3) is None and host.matrix_tables([], None, 0) is None
    q, w = torch.zeros(1, 2, 1, 3, 16, dtype=torch.bfloat16), torch.ones(16)
    assert T.qk_norm_shape(q.shape, w).D == 16
    with pytest.raises(ValueError):  # the general path says what is wrong: not on a GPU
        T.triattn_qk_norm_fwd(q, q, w, w)
    with pytest.raises(ValueError):
        T.triattn_relpos_fwd(torch.zeros(65, 4), torch.zeros(1, 4, 9, 9, dtype=torch.bfloat16))


def test_not_an_extension(fresh, tmp_path):
    p = tmp_path / "host.so"
    p.write_bytes(b"of another machine")
    fresh.setattr(B, "host_path", lambda: str(p))
    with pytest.warns(RuntimeWarning, match="native part"):
        T.load()
    assert T._host() is T._General


def test_there(fresh):
    T.load()
    assert T._host() is not T._General


def test_its_name_is_of_one_torch_and_one_python():
    name = os.path.basename(B.host_path())
    assert torch.__version__ in name and sysconfig.get_config_var("SOABI") in name


def test_the_library_is_built_without_it(monkeypatch):
    B.build()

    def fails(*a):
        raise RuntimeError("no headers")
    monkeypatch.setattr(B, "_build_host", fails)
    with pytest.warns(RuntimeWarning, match="no headers"):
        assert B.build() == B.lib_path() and os.path.exists(B.lib_path())


def test_what_does_not_compile_leaves_no_older_one(monkeypatch, tmp_path):
    p = tmp_path / "host.so"
    p.write_bytes(b"older")
    monkeypatch.setattr(B, "host_path", lambda: str(p))
    monkeypatch.setattr(B, "INCLUDE", str(tmp_path))  # no triattn.h
    (tmp_path / "triattn.h").write_text("#error none\n")
    with pytest.raises(RuntimeError):
        B._build_host(True, False)
    assert not p.exists()
