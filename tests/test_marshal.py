"""The compiled marshalling without a GPU: it leaves every call that is not as it should be to the Python."""
import os
import sys

import pytest

import dense_gemm_preshuffle_amd as gp


def test_host_tensors_and_wrong_counts_are_left():
    import torch

    m = gp._compiled()
    assert m is not None, "not built"
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    assert m.norm(gp.GP_BF16, x, None, 1.0, 0, None, None, None, 1, None, None, 1e-6, True, None, None, 0, 0) is None
    assert m.norm(gp.GP_BF16, x) is None and m.norm() is None
    assert m.linear(gp.GP_BF16, x, x, None, 0, None, False, None, None, None, 0, 0) is None
    assert m.linear(gp.GP_BF16, None, None, None, 0, None, False, None, None, None, 0, 0) is None
    assert m.linear("a", "b", "c", None, 0, None, False, None, None, None, 0, 0) is None
    assert m.norm_backward(*([None] * 22)) is None and m.linear_backward(*([None] * 15)) is None
    with pytest.raises(TypeError):
        m.bind(1, 2)


class _Module:
    """Stands in for a module that was built from other sources; None: one that does not say from which."""

    def __init__(self, sources):
        if sources is not None:
            self.sources = sources
        self.bound = []

    def bind(self, *addresses):
        self.bound.append(addresses)


@pytest.fixture
def fresh():
    gp._compiled.cache_clear()
    yield
    gp._compiled.cache_clear()


@pytest.mark.parametrize("sources", [None, "", "0" * 64])
def test_a_module_of_other_sources_is_not_used(monkeypatch, fresh, sources):
    """One that was compiled against another header would call the entry points through other signatures."""
    other = _Module(sources)
    monkeypatch.setitem(sys.modules, "dense_gemm_preshuffle_amd._marshal", other)
    monkeypatch.setattr(gp, "_marshal", other, raising=False)
    with pytest.warns(UserWarning, match="other sources"):
        assert gp._compiled() is None
    assert not other.bound


def test_a_module_of_these_sources_is_used(monkeypatch, fresh):
    same = _Module(gp.marshal_hash())
    monkeypatch.setitem(sys.modules, "dense_gemm_preshuffle_amd._marshal", same)
    monkeypatch.setattr(gp, "_marshal", same, raising=False)
    assert gp._compiled() is same and len(same.bound[0]) == 7


def test_what_a_module_is_built_from(monkeypatch, tmp_path):
    """The hash follows the marshalling, the header and torch; the built module has it."""
    import torch

    pkg = tmp_path / "p"
    (pkg / "csrc").mkdir(parents=True)
    (tmp_path / "include").mkdir()
    for f in ("csrc/marshal.cpp", "../include/gemm_preshuffle.h"):
        (pkg / f).write_bytes(open(os.path.join(os.path.dirname(gp.__file__), f), "rb").read())
    monkeypatch.setattr(gp, "_PKG", str(pkg))
    now = gp.marshal_hash()
    seen = {now}
    for f in ("csrc/marshal.cpp", "../include/gemm_preshuffle.h"):
        was = (pkg / f).read_bytes()
        (pkg / f).write_bytes(was + b"\n")
        seen.add(gp.marshal_hash())
        (pkg / f).write_bytes(was)
    assert gp.marshal_hash() == now and len(seen) == 3
    monkeypatch.setattr(torch, "__version__", "0.0")
    assert gp.marshal_hash() not in seen
    monkeypatch.undo()
    assert gp._compiled().sources == gp.marshal_hash() == now
