"""The build itself, on a library of one small source file in a folder of its own."""
import os
import subprocess
import sys
import textwrap

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(folder, script):
    head = f"""
        import os, sys
        sys.path.insert(0, {ROOT!r})
        from sparse_embedding_bag_gb300 import build as B
        B.CSRC = {str(folder)!r}
        B.BUILD, B.LIB, B.ENTRY = (os.path.join(B.CSRC, n) for n in ("_build", "lib.so", "_entry.so"))
        B.ENTRY_SRC = os.path.join(B.CSRC, "entry.cpp")
    """
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(head) + textwrap.dedent(script)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_the_library_builds_without_pytorch(tmp_path):
    (tmp_path / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (tmp_path / "entry.cpp").write_text("#error needs PyTorch\n")
    run(tmp_path, """
        import ctypes
        sys.modules["torch"] = None  # importing it fails
        assert B.build() == B.LIB and ctypes.CDLL(B.LIB).one() == 1 and not os.path.exists(B.ENTRY)
        before = os.path.getmtime(B.LIB)
        B.build()
        assert os.path.getmtime(B.LIB) == before
    """)
