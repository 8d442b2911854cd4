"""What qg_device_status costs a program that never calls the cached decode, and that it still sees
those calls' words once it has."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import time
import torch
import gguf_block_dequant_gb300 as qg
qg.load()
torch.zeros(1, device="cuda")

def cost():
    best = 1.0
    for _ in range(300):
        t = time.perf_counter()
        assert qg.device_status() == 0
        best = min(best, time.perf_counter() - t)
    return best * 1e6

before = cost()
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
pool = torch.zeros((2, 8, 16, 2, 64), dtype=torch.float16, device="cuda")
cache = qg.kv_cache(pool[0], pool[1])
batch = qg.kv_batch(i32([100]), i32([[0, 1, 2, 3, 4, 5, 6]]), i32([0, 100]), 100)
x = torch.zeros((100, 12 * 64), device="cuda")
q = torch.zeros((100, 8, 64), dtype=torch.float16, device="cuda")
out = torch.empty((100, 8, 64), device="cuda")
qg.kv_append(cache, batch, x[:, :512], x[:, 512:640], x[:, 640:], q, qg.rope_freqs(64, 1e4).cuda())
qg.attn_paged(cache, batch, q, out, 0.1, torch.empty(qg.attn_workspace_size(cache, batch, 8), dtype=torch.uint8, device="cuda"))
print(before, cost())
batch = qg.kv_batch(i32([100]), i32([[0, 1, 2, 3, 4, 5, 9]]), i32([0, 100]), 100)
qg.kv_append(cache, batch, x[:, :512], x[:, 512:640], x[:, 640:], q, None)
assert qg.device_status() == 1 << qg.QG_EDEVICE_ID
"""


def test_status_words_are_asked_for_once_they_can_be_set():
    """Ten words take ten copies from the device, seven take seven: the least time of 300 calls before
    and after the first cached-decode calls of a process (91 and 126 us on a GB300)."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gguf_block_dequant_gb300 import build

    build.build()
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    before, after = map(float, r.stdout.split())
    assert before < 0.9 * after, (before, after)
