"""Several processes that build the library at once, with a compiler stood in for."""
import os
import subprocess
import sys
import textwrap

MODULE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "farthest_point_sampling_b200", "_build.py")

NVCC = """#!{python}
import os, sys, time
args = sys.argv[1:]
out = args[args.index("-o") + 1]
inputs = [a for a in args if a.endswith(".o") and a != out] if "-c" not in args else [args[args.index("-c") + 1]]
time.sleep(0.02)
data = b"".join(open(p, "rb").read() for p in inputs)  # an object that is gone fails here
with open({log!r}, "a") as f:
    f.write(("compile " if "-c" in args else "link ") + os.path.basename(inputs[0]) + "\\n")
open(out, "wb").write(data)
"""

CHILD = """
import importlib.util, sys
spec = importlib.util.spec_from_file_location("build_module", {module!r})
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
at = {at!r}
print("ready", flush=True)
b.HERE, b.CSRC, b.INCLUDE = at, at + "/csrc", at + "/include"
b.LIB, b.OBJ = at + "/lib.so", at + "/_build"
sys.stdin.readline()
print(b.build(force=len(sys.argv) > 1))
"""


def _run(tmp_path, children, *args):
    log = str(tmp_path / "log")
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(NVCC.format(python=sys.executable, log=log))
    nvcc.chmod(0o755)
    code = textwrap.dedent(CHILD.format(module=MODULE, at=str(tmp_path)))
    procs = [subprocess.Popen([sys.executable, "-c", code, *args], stdin=subprocess.PIPE, stdout=subprocess.PIPE, stderr=subprocess.PIPE,
                              text=True, env={**os.environ, "NVCC": str(nvcc)}) for _ in range(children)]
    for p in procs:
        assert p.stdout.readline() == "ready\n"
    for p in procs:
        p.stdin.write("go\n")
        p.stdin.flush()
    ends = [p.communicate(timeout=120) for p in procs]
    assert all(p.returncode == 0 for p in procs), [e[1][-600:] for e in ends]
    with open(log) as fh:
        made = fh.read().split("\n")[:-1]
    os.remove(log)
    return made


def _tree(tmp_path, version):
    for d in ("csrc", "include"):
        os.makedirs(tmp_path / d, exist_ok=True)
    for i in range(12):
        (tmp_path / "csrc" / f"k{i:02d}.cu").write_text(f"source {i} version {version}\n")
    (tmp_path / "include" / "a.h").write_text("header\n")


def _whole(tmp_path, version):
    assert (tmp_path / "lib.so").read_text() == "".join(f"source {i} version {version}\n" for i in range(12))
    left = sorted(os.listdir(tmp_path / "_build"))
    assert len([n for n in left if n.endswith(".o")]) == 12 and not [n for n in left if ".tmp" in n]


def test_processes_that_build_at_once(tmp_path):
    """All end well, one of them compiles, and objects of older sources go."""
    for version in range(3):
        _tree(tmp_path, version)
        if version:
            os.utime(tmp_path / "lib.so", (1, 1))
        made = _run(tmp_path, 4)
        assert len([m for m in made if m.startswith("compile")]) == 12 and len([m for m in made if m.startswith("link")]) == 1
        _whole(tmp_path, version)


def test_forced_builds_at_once(tmp_path):
    _tree(tmp_path, 0)
    for _ in range(2):
        made = _run(tmp_path, 3, "force")
        assert len([m for m in made if m.startswith("compile")]) == 36
        _whole(tmp_path, 0)
