"""The build's resource guard: a kernel that spills registers or keeps an
array in scratch memory fails the build (host-only)."""
import re

import pytest

from dense_gemm_preshuffle_amd import build as B

SAMPLE = """\
./k.hpp:171:1: remark: Function Name: _Z4fastv [-Rpass-analysis=kernel-resource-usage]
./k.hpp:171:1: remark:     VGPRs: 128 [-Rpass-analysis=kernel-resource-usage]
./k.hpp:171:1: remark:     VGPRs Spill: 0 [-Rpass-analysis=kernel-resource-usage]
./k.hpp:171:1: remark:     ScratchSize [bytes/lane]: 0 [-Rpass-analysis=kernel-resource-usage]
./k.hpp:171:1: remark: Function Name: _Z5arrayv [-Rpass-analysis=kernel-resource-usage]
./k.hpp:171:1: remark:     VGPRs: 70 [-Rpass-analysis=kernel-resource-usage]
./k.hpp:171:1: remark:     VGPRs Spill: 0 [-Rpass-analysis=kernel-resource-usage]
./k.hpp:171:1: remark:     ScratchSize [bytes/lane]: 1552 [-Rpass-analysis=kernel-resource-usage]
./k.hpp:171:1: remark: Function Name: _Z5spillv [-Rpass-analysis=kernel-resource-usage]
./k.hpp:171:1: remark:     VGPRs Spill: 20 [-Rpass-analysis=kernel-resource-usage]
./k.hpp:171:1: remark:     ScratchSize [bytes/lane]: 68 [-Rpass-analysis=kernel-resource-usage]
"""


def test_resource_remarks_parsed():
    res = B.kernel_resources(SAMPLE)
    assert set(res) == {"_Z4fastv", "_Z5arrayv", "_Z5spillv"}
    assert res["_Z4fastv"]["VGPRs"] == "128"


def test_scratch_and_spills_flagged():
    bad = dict(B.spilling(B.kernel_resources(SAMPLE)))
    assert set(bad) == {"_Z5arrayv", "_Z5spillv"}
    assert bad["_Z5arrayv"] == [0, 0, 1552] and bad["_Z5spillv"] == [20, 0, 68]


def _dry(monkeypatch, tmp_path):
    """The build with its compilers replaced by files that say what they are."""
    import subprocess

    for name in ("BUILD", "LIB", "PROBE_LIB", "MARSHAL"):
        monkeypatch.setattr(B, name, str(tmp_path / name))
    monkeypatch.setattr(B, "_sources", lambda: ["a.hip"])
    monkeypatch.setattr(B, "_compile", lambda src: (src + ".o", {}))

    def run(cmd, **kw):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("linked")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(B.subprocess, "run", run)
    (tmp_path / "MARSHAL").write_text("of an earlier build")


@pytest.mark.parametrize("error", [RuntimeError("marshal.cpp failed"), ImportError("no torch"), FileNotFoundError("g++")])
def test_the_library_is_built_without_the_marshalling(monkeypatch, tmp_path, error):
    """Calls go without the module, so what stops its build stops nothing else; an older module does not stay."""
    _dry(monkeypatch, tmp_path)

    def fail():
        raise error
    monkeypatch.setattr(B, "build_marshal", fail)
    with pytest.warns(UserWarning, match=re.escape(str(error))):
        lib = B.build(jobs=2)
    assert lib == str(tmp_path / "LIB") and (tmp_path / "LIB").read_text() == (tmp_path / "PROBE_LIB").read_text() == "linked"
    assert not (tmp_path / "MARSHAL").exists()


def test_the_marshalling_is_kept_where_it_is_built(monkeypatch, tmp_path):
    _dry(monkeypatch, tmp_path)
    monkeypatch.setattr(B, "build_marshal", lambda: (tmp_path / "MARSHAL").write_text("new"))
    B.build(jobs=2)
    assert (tmp_path / "MARSHAL").read_text() == "new"
