"""The compiled part of the binding and other Python threads: they run while a call waits in
the library, and several may be in it at once.  (A call waits for its stream where
LF_DEBUG_SYNC is set, which is read once per process, so that check runs in a child process;
the stream is held up by a kernel that ends by itself.)"""
import os
import subprocess
import sys
import threading

import pytest
import torch

import layout_folding_gb300 as lf
from layout_folding_gb300 import compiled

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import sys, threading, time
sys.path.insert(0, %r)
import torch
import layout_folding_gb300 as lf
from layout_folding_gb300 import compiled
torch.cuda.set_device(0)
assert compiled.load() is not None
x = torch.randn(64, 64, device="cuda").bfloat16()
w = torch.randn(64, device="cuda").bfloat16()
calls = [lambda: lf.linear(x, x), lambda: lf.linear_backward(x, x, x), lambda: lf.block_norm(x, x, w, w),
         lambda: lf.block_norm_backward(x, x, x, w, w)]
for call in calls:
    call()
assert all("built-in" in repr(getattr(compiled, name)) for name in compiled._NAMES)
longest, done = 0.0, False
def tick():
    global longest
    last = time.perf_counter()
    while not done:
        time.sleep(0.001)
        now = time.perf_counter()
        longest, last = max(longest, now - last), now
thread = threading.Thread(target=tick, daemon=True)
thread.start()
time.sleep(0.05)
for call in calls:
    torch.cuda.synchronize()
    longest = 0.0
    lf.occupy_sms(1, 400_000_000)
    began = time.perf_counter()
    call()
    waited = time.perf_counter() - began
    time.sleep(0.01)
    print("waited %%.3f s, the other thread at most %%.3f s" %% (waited, longest))
    assert waited > 0.3 and longest < 0.2, (waited, longest)
done = True
thread.join()
print("threads ok")
''' % ROOT


def test_other_threads_run_while_a_call_waits():
    env = dict(os.environ, LF_DEBUG_SYNC="1")
    r = subprocess.run([sys.executable, "-c", CHILD], env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "threads ok" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


def test_several_threads_at_once():
    assert compiled.load() is not None
    torch.cuda.set_device(0)
    g = torch.Generator().manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g).bfloat16().cuda()
    x, w, weight, dy = normal(300, 264), normal(136, 264), normal(264), normal(300, 136)

    def all_calls():
        out, pre = lf.linear(x, w, act="gelu", want_pre=True)
        return (out, pre, *lf.linear_backward(dy, x, w, pre=pre, act="gelu")[:2], *lf.block_norm(x, x, weight, weight)[:2],
                *lf.block_norm_backward(x, x, x, weight, weight)[:4])
    want = [t.clone() for t in all_calls()]
    torch.cuda.synchronize()
    wrong = []

    def work():
        torch.cuda.set_device(0)
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    got = all_calls()
                    wrong.extend(i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b))
        except Exception as e:  # (a thread's own exception would not fail the test)
            wrong.append(e)
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    lf.check_device_error()
    assert not wrong, wrong[:5]
