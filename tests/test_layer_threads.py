"""The calls of bcjr_layer.h from several host threads (CPU only: the library over a stand-in for the CUDA runtime).

A kernel's limit of dynamic shared memory belongs to the process, while each launch needs another size; a thread
that sets it between another one's setting and its launch must not leave it too low."""
import json
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

# runs in a process of its own, where the stand-in's symbols come before the runtime's
PROGRAM = r"""
import ctypes, sys, threading
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
P, I = ctypes.c_void_p, ctypes.c_int
lib.bcjr_int4_matmul.argtypes = [P, I, I, I, I, P, P, I, P, I, P, P]
lib.bcjr_trellis_matmul.argtypes = [P, I, I, I, I, P, P, I, I, I, I, P, I, P, P]

def int4(tokens, cols, kind=2):
    return lib.bcjr_int4_matmul(1 << 20, kind, tokens, 64, cols, 1 << 24, 1 << 28, 0, None, 128, 1 << 30, None)

def trellis(tokens, L, kind=0):
    return lib.bcjr_trellis_matmul(1 << 20, kind, tokens, 64, 4096, 1 << 24, 1 << 28, kind, L, 2, 256, None, 0, 1 << 30, None)

# (small, large) needs of one kernel: columns staged at a time, tokens staged, copies of the codebook, one held half
PAIRS = {
    "int4": (lambda: int4(1, 256), lambda: int4(4, 16384)),
    "int4 rows": (lambda: int4(6, 256, 0), lambda: int4(10, 16384, 0)),
    "int4 rows 16 bits": (lambda: int4(17, 256), lambda: int4(32, 16384)),
    "trellis": (lambda: trellis(1, 4), lambda: trellis(1, 15)),
    "trellis several": (lambda: trellis(3, 4), lambda: trellis(3, 15)),
}
HOOK = ctypes.CFUNCTYPE(None)
what = sys.argv[3]
if what in PAIRS:
    small, large = PAIRS[what]
    other = []
    hook = HOOK(lambda: other.append(small()))
    fake.fake_after_set(hook)
    first = large()
    print([first, other, large(), small(), large(), fake.fake_refused()])
elif what == "threads":
    bad = []
    def work(seed):
        for i in range(400):
            for n, pair in enumerate(PAIRS.values()):
                status = pair[(seed + i + n) % 2]()
                if status:
                    bad.append(status)
    threads = [threading.Thread(target=work, args=(s,)) for s in range(8)]
    for t in threads: t.start()
    for t in threads: t.join()
    print([bad[:5], fake.fake_refused(), fake.fake_launches()])
else:  # a limit that could not be raised is asked for again
    fake.fake_fail_sets(1)
    print([PAIRS["trellis"][1](), PAIRS["trellis"][1](), fake.fake_refused()])
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    from differentiable_bcjr_b200 import build
    gcc = shutil.which("gcc")
    include = next((d for d in (os.path.join(os.environ.get("CUDA_HOME", ""), "include"), "/usr/local/cuda/include")
                    if os.path.exists(os.path.join(d, "cuda_runtime_api.h"))), None)
    if not gcc or not include:
        pytest.skip("needs gcc and the CUDA headers")
    so = str(tmp_path_factory.mktemp("fake") / "fake.so")
    subprocess.run([gcc, "-shared", "-fPIC", "-O1", "-I", include, os.path.join(HERE, "fake_cudart.c"), "-o", so], check=True)
    lib = build.build()

    def go(what):
        out = subprocess.run([sys.executable, "-c", PROGRAM, so, lib, what], check=True, capture_output=True, text=True, timeout=120).stdout
        return json.loads(out)

    return go


@pytest.mark.parametrize("what", ["int4", "int4 rows", "int4 rows 16 bits", "trellis", "trellis several"])
def test_a_smaller_launch_in_between_leaves_the_limit(run, what):
    assert run(what) == [0, [0], 0, 0, 0, 0]


def test_eight_threads_of_all_sizes(run):
    bad, refused, launches = run("threads")
    assert not bad and refused == 0 and launches == 8 * 400 * 5


def test_a_limit_that_was_refused_is_asked_for_again(run):
    assert run("failing") == [4, 0, 0]  # BCJR_ERR_CUDA, once
