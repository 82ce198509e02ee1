"""The build: what it compiles with and without torch, and when the binding
counts as up to date.  Compilers are stood in for by a function that writes the files
they would; each case is a process of its own."""
import os
import subprocess
import sys
import textwrap

BUILD = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_activation_quantization_bsq_gb300", "_build.py")
START = """
import importlib.util, os, subprocess, sys, sysconfig
{before}
spec = importlib.util.spec_from_file_location("the_build", sys.argv[1])
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
into = b.LIB_DIR
for name, value in list(vars(b).items()):
    if isinstance(value, str) and value.startswith(into):
        setattr(b, name, sys.argv[2] + value[len(into):])
ran = []
class Compiler:
    returncode, stdout, stderr = 0, "", ""
    def __init__(self, command, **kw):
        ran.append(command)
        out = command[command.index("-o") + 1]
        if out != os.devnull:
            open(out, "w").close()
    def communicate(self):
        return "", None
b.subprocess = type("S", (), dict(Popen=Compiler, run=Compiler, PIPE=None, STDOUT=None))
b.nvcc_path = lambda: "/usr/local/cuda/bin/nvcc"
made = lambda: sorted(f for f in os.listdir(sys.argv[2]) if f.endswith(".so"))
"""


def run(tmp_path, script, before="", path=None):
    env = dict(os.environ)
    if path is not None:
        env["PYTHONPATH"] = str(path)
    lib = tmp_path / "lib"
    lib.mkdir(exist_ok=True)
    done = subprocess.run([sys.executable, "-c", START.format(before=before) + textwrap.dedent(script), BUILD, str(lib)], capture_output=True, text=True,
                          env=env, cwd=tmp_path)
    assert done.returncode == 0, done.stderr


def test_the_library_builds_without_torch(tmp_path):
    run(tmp_path, """
        assert b.is_stale()
        assert b.build() == b.LIB_PATH
        assert made() == ["libbsq.so"], made()
        assert all(any(c[-1].endswith(s) for c in ran) for s in b.SOURCES)
        assert not any("torch" in a for c in ran for a in c)
        assert not b.is_stale()
    """, before="sys.modules['torch'] = None")   # as where it is not installed


def test_a_binding_of_another_torch_is_not_up_to_date(tmp_path):
    """Compiled against one torch, the binding is neither found nor taken as up to date with another version, or another Python."""
    for version in ("2.11.0+cu130", "2.12.0"):
        package = tmp_path / version / "torch"
        package.mkdir(parents=True)
        (package / "__init__.py").write_text("")
        (package / "version.py").write_text(f"from typing import Optional\n__all__ = ['__version__']\n__version__ = '{version}'\ndebug = False\n")
    build = """
        assert b.is_stale()
        b.build()
        assert not b.is_stale() and os.path.exists(b.BINDING_PATH)
        assert any("torch" in a for c in ran for a in c)
    """
    run(tmp_path, build, path=tmp_path / "2.11.0+cu130")
    run(tmp_path, "assert not b.is_stale()", path=tmp_path / "2.11.0+cu130")
    run(tmp_path, build, path=tmp_path / "2.12.0")
    run(tmp_path, "assert not b.is_stale()", path=tmp_path / "2.12.0")
    run(tmp_path, "assert b.is_stale() and not os.path.exists(b.BINDING_PATH)", path=tmp_path / "2.12.0",
        before="sysconfig.get_config_vars()['EXT_SUFFIX'] = '.cpython-399-other.so'")
