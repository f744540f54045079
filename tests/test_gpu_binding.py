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


def test_threads_with_streams_of_their_own():
    """Four threads call at once, each on its stream and its cache: every result
    is the one that the same calls give alone."""
    import threading

    def work(seed, stream):
        with torch.cuda.stream(stream):
            g = torch.Generator(device="cuda").manual_seed(seed)
            B, Hq, Hkv, d, page, M = 5 + 60 * (seed % 2), 8, 2, 64, 16, 700
            pools = [torch.zeros((B * 8, page, Hkv, d), dtype=torch.uint8, device="cuda")
                     for _ in "kv"]
            scales = [torch.zeros((B * 8, Hkv), device="cuda") for _ in "kv"]
            table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
            table[:, :8] = torch.arange(B * 8, device="cuda").reshape(B, 8)
            lens = torch.zeros(B, dtype=torch.int32, device="cuda")
            freqs = dsa.rope_freqs(d)[0]
            idx = torch.arange(16, dtype=torch.int32, device="cuda").repeat(B, 1)
            err = dsa.error_word()
            out = []
            for step in range(40):
                x = torch.randn((B, Hq + 2 * Hkv, d), generator=g, device="cuda").bfloat16()
                q, k = dsa.rope(x[:, :Hq], x[:, Hq:Hq + Hkv], lens.long(), freqs)
                dsa.kv8_append(k, x[:, Hq + Hkv:], *pools, *scales, table, lens, err=err)
                lens = lens + 1
                O = dsa.attn_kv8(q, *pools, *scales, table, lens, 0.125, err=err)
                rows = torch.where(idx < lens[:, None], idx, -1)
                S = dsa.sparse_attn_kv8(O, *pools, *scales, table, lens, rows, 0.125, err=err)
                out += [O, S]
            out += pools + scales
            stream.synchronize()
            assert dsa.device_error(err=err) == dsa.DEVERR_NONE
            return out

    want = [work(seed, torch.cuda.Stream()) for seed in range(4)]
    got, failed = [None] * 4, []

    def run(seed):
        try:
            got[seed] = work(seed, torch.cuda.Stream())
        except BaseException as e:
            failed.append(e)

    for _ in range(3):
        threads = [threading.Thread(target=run, args=(seed,)) for seed in range(4)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not failed
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
