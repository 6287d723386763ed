"""An exception that ends a thread of a test fails the test: the threaded tests' workers only report results that differ."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

BAD = """
import threading

def test_threads():
    failed = []

    def work():
        raise RuntimeError("a launch that failed")

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not failed
"""


def _run(tmp_path, text):
    (tmp_path / "test_threads.py").write_text(text)
    return subprocess.run([sys.executable, "-m", "pytest", "-q", "-c", os.path.join(ROOT, "pytest.ini"), "--rootdir", str(tmp_path), str(tmp_path)],
                          capture_output=True, text=True, cwd=tmp_path)


def test_a_thread_that_raises_fails_its_test(tmp_path):
    r = _run(tmp_path, BAD)
    assert r.returncode == 1 and "a launch that failed" in r.stdout, r.stdout


def test_a_thread_that_ends_does_not(tmp_path):
    r = _run(tmp_path, BAD.replace('raise RuntimeError("a launch that failed")', "pass"))
    assert r.returncode == 0, r.stdout
