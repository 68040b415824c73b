"""The calls of bcjr_layer.h from several host threads at once, and captured before any of them ever ran (needs a B200)."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _calls():
    """Calls of one kernel each that need little and much shared memory, and the other calls beside them."""
    import differentiable_bcjr_b200 as B
    gen = torch.Generator().manual_seed(1)
    out = []
    for kind in (F32, BF16):
        for tokens in (1, 2, 17):
            for cols in (256, 8192):
                packed, scales, zeros = B.int4_quantize(torch.randn(64, cols, generator=gen).cuda(), 128, True)
                x = torch.randn(tokens, cols, generator=gen).to(kind).cuda()
                out.append(lambda x=x, a=(packed, scales, zeros): B.int4_matmul(x, *a, 128))
            for L in (4, 12, 15, 16):
                states = R.random_path(64 * 4, 128, L, 2, L).cuda()
                stream, c = B.trellis_pack(states, L, 2), torch.randn(1 << L, generator=gen).to(kind).cuda()
                x = torch.randn(tokens, 512, generator=gen).to(kind).cuda()
                out.append(lambda x=x, s=stream, c=c, L=L: B.trellis_matmul(x, s, c, L, 2, 128))
                out.append(lambda s=states, L=L: B.trellis_pack(s, L, 2))
    w = torch.randn(300, 1000, generator=gen).cuda()
    for group in (32, 128, 0):
        out.append(lambda g=group: B.int4_quantize(w, g)[0])
    for bits in (8, 32):
        def adamw(bits=bits):
            p, g = w.clone(), w * 0.1
            state = B.adamw_state([p], bits)
            B.adamw_step([p], [g], state[0], state[1], 1, scales=state[2])
            return p
        out.append(adamw)
    return out


def test_threads_on_streams_of_their_own():
    calls = _calls()
    want = [f() for f in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(seed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                order = torch.randperm(len(calls), generator=torch.Generator().manual_seed(seed)).tolist()
                for _ in range(5):
                    got = [(i, calls[i]()) for i in order]
                    torch.cuda.current_stream().synchronize()
                    wrong.extend(i for i, y in got if not torch.equal(y.view(torch.uint8), want[i].view(torch.uint8)))
        except Exception as e:  # noqa: BLE001 (to the test's own thread)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:5]


PROGRAM = """
import sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import torch
import layer_ref as R
import differentiable_bcjr_b200 as B
gen = torch.Generator().manual_seed(1)
w, x = torch.randn(64, 512, generator=gen).cuda(), torch.randn(3, 512, generator=gen).cuda()
states, c = R.random_path(256, 128, 15, 2, 1).cuda(), torch.randn(1 << 15, generator=gen).cuda()
p, g = w.clone(), w * 0.1
state, count = B.adamw_state([p], 8), torch.ones(1, dtype=torch.int64, device="cuda")

def all_of_them():
    B.adamw_step([p], [g], state[0], state[1], count, scales=state[2])
    return (B.int4_matmul(x, *B.int4_quantize(w, 128), 128), B.trellis_matmul(x, B.trellis_pack(states, 15, 2), c, 15, 2, 128),
            B.trellis_matmul(x.bfloat16(), B.trellis_pack(states, 15, 2), c.bfloat16(), 15, 2, 128))

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = all_of_them()
graph.replay()
first = p.clone()
again = [t.clone() for t in y]
for t in (p, *state):
    t.view(torch.uint8).zero_()
p.copy_(w)
want = all_of_them()
assert all(torch.equal(a, b) for a, b in zip(again, want)) and torch.equal(first, p)
print("same")
"""


def test_capture_of_first_calls():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
