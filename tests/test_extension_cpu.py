"""The extension of the attention calls belongs to one Python (no GPU needed)."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

moe = pytest.importorskip("block_scaled_fp4_group_amd")


def test_the_extension_has_this_pythons_tag():
    assert os.path.basename(moe._calls.__file__) == "_calls" + sysconfig.get_config_var("EXT_SUFFIX")
    assert not os.path.exists(os.path.join(os.path.dirname(moe.__file__), "_calls.so"))


@pytest.mark.parametrize("other", ["_calls.so", "_calls.cpython-399-x86_64-linux-gnu.so", None])
def test_another_pythons_extension_is_not_loaded(tmp_path, other):
    """The package then says that its own is not built."""
    src, dst = os.path.dirname(moe.__file__), tmp_path / "block_scaled_fp4_group_amd"
    dst.mkdir()
    for f in os.listdir(src):
        if f.endswith(".py"):
            shutil.copy(os.path.join(src, f), dst)
    (dst / "libmoefp4.so").symlink_to(os.path.join(src, "libmoefp4.so"))
    if other:
        (dst / other).symlink_to(moe._calls.__file__)
    r = subprocess.run([sys.executable, "-c", "import block_scaled_fp4_group_amd"], capture_output=True, text=True, cwd=tmp_path)
    assert r.returncode == 1 and "is not built; run" in r.stderr and "ImportError" in r.stderr


def test_hipcc_builds_everything(tmp_path, monkeypatch):
    """No other compiler is asked for; without Python's headers the build says so."""
    import importlib.util
    spec = importlib.util.spec_from_file_location("_build", os.path.join(os.path.dirname(moe.__file__), "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    for command in (build.compile_command("a.hip", "a.o"), build.link_command(["a.o"], "a.so"), build.calls_command("c.so")):
        assert command[0] == build.hipcc()
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    with pytest.raises(RuntimeError, match="Python's headers"):
        build.calls_command("c.so")
