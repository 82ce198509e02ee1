"""The build: what it compiles with and without torch, and when the binding
counts as up to date.  Compilers are stood in for by a function that writes the files
they would; each case is a process of its own."""
import os
import subprocess
import sys
import textwrap

BUILD = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_activation_quantization_bsq_gb300", "_build.py")
START = """
import importlib.util, os, subprocess, sys
spec = importlib.util.spec_from_file_location("the_build", sys.argv[1])
if {hidden}:
    sys.modules["torch"] = None          # as where torch is not installed
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


def run(tmp_path, script, hidden=False, path=None):
    env = dict(os.environ)
    if path is not None:
        env["PYTHONPATH"] = str(path)
    lib = tmp_path / "lib"
    lib.mkdir(exist_ok=True)
    done = subprocess.run([sys.executable, "-c", START.format(hidden=hidden) + textwrap.dedent(script), BUILD, str(lib)], capture_output=True, text=True,
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
    """, hidden=True)
