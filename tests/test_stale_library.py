"""The binding and a library that was built before some calls were added."""
import os
import shutil
import subprocess

import pytest

from sparse_mixture_experts_renormalised_amd import binding


@pytest.mark.parametrize("version", ["MOE_VERSION", "0x000100"])
def test_a_library_without_some_calls_is_refused_by_name(tmp_path, monkeypatch, version):
    """Calls that are added do not change MOE_VERSION, so an older library passes for
    the same interface: what it lacks is named, and so is another version, before any
    symbol of this one is asked for."""
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src, so = tmp_path / "old.c", tmp_path / "old.so"
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    src.write_text(f'#include "moe_mi355x.h"\nint moe_version(void) {{ return {version}; }}\n')
    subprocess.run([cc, "-shared", "-fPIC", "-I", include, str(src), "-o", str(so)], check=True)
    monkeypatch.setattr(binding, "LIB_PATH", str(so))
    monkeypatch.setattr(binding, "_LIB", None)
    with pytest.raises(RuntimeError, match="rebuild the library") as e:
        binding.lib()
    assert ("moe_route" in str(e.value)) == (version == "MOE_VERSION")


def test_a_file_that_is_no_such_library(tmp_path, monkeypatch):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src, so = tmp_path / "none.c", tmp_path / "none.so"
    src.write_text("int other(void) { return 0; }\n")
    subprocess.run([cc, "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    monkeypatch.setattr(binding, "LIB_PATH", str(so))
    monkeypatch.setattr(binding, "_LIB", None)
    with pytest.raises(RuntimeError, match="moe_version.*rebuild the library"):
        binding.lib()
