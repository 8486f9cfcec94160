"""The build by itself, in a folder of its own and with one source file (no GPU)."""
import os
import subprocess
import sys

BUILD = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "q4_quantized_matmul_gb300", "build.py")

# loads build.py as a file, its outputs in argv[1] and q4q_noalloc.cu its only source
SET_UP = """
import importlib.util, os, sys
spec = importlib.util.spec_from_file_location("q4q_build", %r)
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.OUT_DIR = sys.argv[1]
b.LIB, b.EXT = os.path.join(sys.argv[1], "libq4q.so"), os.path.join(sys.argv[1], "_q4q_torch.so")
one = os.path.join(b.CSRC, "q4q_noalloc.cu")
b._sources = lambda: [one]
""" % BUILD

# what a machine without torch does: no module of that name is found
NO_TORCH = """
class Absent:
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ModuleNotFoundError("No module named 'torch'", name="torch")
sys.meta_path.insert(0, Absent())
found = importlib.util.find_spec
importlib.util.find_spec = lambda name, package=None: None if name.split(".")[0] == "torch" else found(name, package)
"""


def run(tmp_path, *parts):
    return subprocess.run([sys.executable, "-c", "".join((SET_UP,) + parts), str(tmp_path)], capture_output=True, text=True, timeout=600)


def test_library_builds_without_torch(tmp_path):
    r = run(tmp_path, NO_TORCH, "\nprint(b.build())\nassert b.up_to_date()\n")
    assert r.returncode == 0, r.stderr[-2000:]
    assert os.path.exists(os.path.join(tmp_path, "libq4q.so")) and not os.path.exists(os.path.join(tmp_path, "_q4q_torch.so"))


def test_library_is_there_when_the_python_side_fails(tmp_path):
    r = run(tmp_path, "\nb.EXT_SRC = os.path.join(sys.argv[1], 'absent.cpp')\nb.build()\n")
    assert r.returncode != 0 and "absent.cpp" in r.stderr
    assert os.path.exists(os.path.join(tmp_path, "libq4q.so")) and not os.path.exists(os.path.join(tmp_path, "_q4q_torch.so"))


def test_python_side_of_another_torch_is_not_up_to_date(tmp_path):
    """The extension is compiled against one torch and one interpreter; file times do not tell them apart."""
    r = run(tmp_path, "\nb.build()\nassert b.up_to_date()\n")
    assert r.returncode == 0, r.stderr[-2000:]
    # in a new process, which has torch not loaded yet, a torch of another version comes first
    r = run(tmp_path, """
assert b.up_to_date()
fake = os.path.join(sys.argv[1], "torch")
os.makedirs(fake)
text = open(os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "version.py")).read()
open(os.path.join(fake, "__init__.py"), "w").close()
open(os.path.join(fake, "version.py"), "w").write(text.replace("__version__ = '", "__version__ = '0"))
sys.path.insert(0, sys.argv[1])
importlib.invalidate_caches()
assert os.path.dirname(importlib.util.find_spec("torch").origin) == fake
assert not b.up_to_date()
""")
    assert r.returncode == 0, r.stderr[-2000:]
