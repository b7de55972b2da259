"""The GPU tests also run from copies of the tree that lack what its ignore
lists name (but for git's own, which names built files): host-only sources and
old records.  Such a copy has to be collected without an error."""
import fnmatch
import glob
import os
import shutil
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def left_out(patterns):
    """For shutil.copytree: './path' names a file or folder from the top, other patterns match at any depth."""
    def names(folder, entries):
        at = os.path.relpath(folder, ROOT)
        out = set()
        for e in entries:
            path = "./" + os.path.normpath(os.path.join(at, e))
            if any(path == p if p.startswith("./") else fnmatch.fnmatch(e, p) for p in patterns):
                out.add(e)
        return out
    return names


def test_a_copy_without_ignored_files_collects(tmp_path):
    lists = [f for f in glob.glob(os.path.join(ROOT, ".*ignore")) if os.path.basename(f) != ".gitignore"]
    patterns = [line.strip() for f in lists for line in open(f) if line.strip()]
    ignore = left_out(patterns + ["__pycache__"])
    for d in ("tests", "oracle", "synth", "gguf_dequant_matvec_amd", "perf"):
        shutil.copytree(os.path.join(ROOT, d), tmp_path / d, ignore=ignore)
    for f in glob.glob(os.path.join(ROOT, "*.py")):
        shutil.copy(f, tmp_path)
    r = subprocess.run([sys.executable, "-m", "pytest", "tests", "--collect-only", "-q", "-p", "no:cacheprovider"], cwd=tmp_path,
                       capture_output=True, text=True, timeout=300, env=dict(os.environ, PYTHONPATH=str(tmp_path)))
    assert r.returncode == 0 and "error" not in r.stdout.lower().splitlines()[-1], r.stdout + r.stderr
