"""The compiled side of the Python binding with tensors on the GPU: what happens
around the library calls, which host tests cannot reach."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

import sparse_long_context_02_b200 as dsa

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# In the library's place: each call waits up to 5 s for another thread to say go, and fails
# without it.  No kernel runs.
STAND_IN = """
#include <unistd.h>
static volatile int said;
void go(void) { said = 1; }
static int wait_for_it(void) {
    said = 0;
    for (int i = 0; i < 5000 && !said; ++i) usleep(1000);
    return said ? 0 : 1;
}
int dsa_rope(void) { return wait_for_it(); }
int dsa_rope_backward(void) { return wait_for_it(); }
int dsa_kv8_append(void) { return wait_for_it(); }
int dsa_sparse_attn_kv8(void) { return wait_for_it(); }
int dsa_attn_kv8(void) { return wait_for_it(); }
unsigned long dsa_attn_kv8_workspace_size(void) { return 0; }
"""

THREADS = """
import ctypes, sys, threading, time
import torch
import sparse_long_context_02_b200 as dsa
native = dsa._load_native()
go = ctypes.CDLL(sys.argv[1]).go
native.bind(sys.argv[1], dsa._check)
q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
pos = torch.zeros(2, dtype=torch.int64, device="cuda")
f = torch.zeros(32, dtype=torch.int64, device="cuda")
i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
pools = [torch.zeros((4, 16, 2, 64), dtype=torch.uint8, device="cuda") for _ in "kv"]
cache = (*pools, *(torch.zeros((4, 2), device="cuda") for _ in "kv"), i32(2, 3), i32(2))
calls = {
    "rope": lambda: dsa.rope(q, None, pos, f),
    "rope_backward": lambda: dsa.rope_backward(q, None, pos, f),
    "kv8_append": lambda: dsa.kv8_append(q[:, :2].contiguous(), q[:, :2].contiguous(), *cache),
    "sparse_attn_kv8": lambda: dsa.sparse_attn_kv8(q, *cache, i32(2, 8), 0.125),
    "attn_kv8": lambda: dsa.attn_kv8(q, *cache, 0.125),
}
for name, call in calls.items():
    t = threading.Thread(target=lambda: (time.sleep(0.2), go()))
    t.start()
    try:
        call()
        print(name, "ran beside another thread")
    except dsa.DSAError:
        print(name, "held the interpreter")
    t.join()
"""


def test_other_threads_run_during_a_call(tmp_path):
    """The calls release the interpreter lock, as ctypes does for the others: a
    launch that waits for room in a full queue does not stop the threads that
    would feed or empty it."""
    cc = shutil.which("gcc") or shutil.which("cc")
    assert cc is not None
    src, so = tmp_path / "stand_in.c", tmp_path / "stand_in.so"
    src.write_text(STAND_IN)
    subprocess.check_call([cc, "-O1", "-shared", "-fPIC", "-o", str(so), str(src)])
    r = subprocess.run([sys.executable, "-c", THREADS, str(so)], cwd=ROOT, capture_output=True,
                       text=True, timeout=240)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = r.stdout.split("\n")
    assert sum("ran beside another thread" in line for line in lines) == 5, r.stdout


def _rope_args(L=2, H=4, d=64):
    return (torch.zeros((L, H, d), dtype=torch.bfloat16, device="cuda"), None,
            torch.zeros(L, dtype=torch.int64, device="cuda"), dsa.rope_freqs(d)[0])


def test_a_flag_without_a_truth_value_raises_its_own_error():
    class Neither:
        def __bool__(self):
            raise KeyError("neither")

    for call in (dsa.rope, dsa.rope_backward):
        with pytest.raises(KeyError, match="neither"):
            call(*_rope_args(), interleaved=Neither())
    dsa.rope(*_rope_args(), interleaved=True)


def test_out_of_memory_is_torchs_error():
    """An output that does not fit raises what torch.empty raises, which callers
    catch to retry with less."""
    q = torch.empty((1 << 20, 4, 64), dtype=torch.bfloat16, device="cuda")  # 512 MB
    pos = torch.zeros(1 << 20, dtype=torch.int64, device="cuda")
    f = dsa.rope_freqs(64)[0]
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction(
        (torch.cuda.memory_reserved() + (64 << 20)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            dsa.rope(q, None, pos, f)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert dsa.rope(q[:8], None, pos[:8], f)[0].shape == (8, 4, 64)
