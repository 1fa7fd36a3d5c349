"""The rotary, cache and attention calls made for the first time inside CUDA-graph capture, in a
fresh process, and from several host threads at once: every output equals the eager call's, bit
for bit."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMMON = r'''
import sys
import torch
sys.path.insert(0, ROOT)
import gemm_q4_q8_gb300 as qg
from gemm_q4_q8_gb300 import build
build.build()

def make(i):
    """A step of its own cache type, head size, group and columns: (run, outputs)."""
    qtype, kv, heads, d, ps, ncols, lens = (
        (qg.Q8_0, 8, 40, 128, 64, 1, [700, 5000, 1]), (qg.QG_F16, 2, 16, 256, 16, 1, [1000]),
        (qg.QG_F16, 4, 32, 64, 32, 8, [2000, 3, 800, 0]), (qg.Q8_0, 1, 17, 64, 16, 16, [300, 17]),
        (qg.Q8_0, 2, 16, 256, 128, 4, [900, 1234]), (qg.QG_F16, 8, 8, 128, 256, 3, [50] * 30))[i]
    n = len(lens)
    pages = -(-max(lens) // ps) + 1
    g = torch.Generator(device="cuda").manual_seed(i)
    pool = torch.full((n * pages * qg.qkv_page_bytes(qtype, kv, d, ps),), 0xFF, dtype=torch.uint8, device="cuda")
    table = torch.randperm(n * pages, generator=g, device="cuda").to(torch.int32).view(n, pages)
    c = qg.qkv_cache(qtype, pool, table, kv, d, ps)
    plan = qg.qrope_plan(d // 2, interleaved=bool(i % 2))
    pos = torch.tensor([j for m in lens for j in range(m)], dtype=torch.int32, device="cuda")
    seq = torch.tensor([s for s, m in enumerate(lens) for _ in range(m)], dtype=torch.int32, device="cuda")
    rows = torch.randn(len(pos), heads + 2 * kv, d, generator=g, device="cuda")
    last = torch.tensor([max(m - ncols, 0) + t for m in lens for t in range(ncols)], dtype=torch.int32, device="cuda")
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(qg.qattn_workspace_bytes(c, heads, ncols), dtype=torch.uint8, device="cuda")
    out = dict(q=torch.empty(len(pos), heads, d, dtype=torch.float16, device="cuda"),
               turned=torch.empty(len(pos), heads, d, device="cuda"),
               k=torch.empty(n * ncols, kv, d, dtype=torch.float16, device="cuda"),
               v=torch.empty(n * ncols, kv, d, dtype=torch.float16, device="cuda"),
               y=torch.empty(n, ncols, heads, d, dtype=torch.float16, device="cuda"), pool=pool)
    queries = torch.randn(n, ncols, heads, d, generator=g, device="cuda").half()
    def run(stream=None):
        qg.qrope(plan, rows[:, :heads], pos, out["turned"], stream=stream)
        qg.qkv_append(c, rows[:, heads:heads + kv], rows[:, heads + kv:], pos, seq=seq, rope=plan, q=rows[:, :heads],
                      q_out=out["q"], stream=stream)
        qg.qkv_read(c, last, out["k"], out["v"], stream=stream)
        qg.qattn_paged(c, queries, lens_d, out["y"], ws, stream=stream)
    return run, out

def wipe(out):
    for n, t in out.items():
        t.fill_(0xFF if n == "pool" else 7)
'''

CAPTURE = r'''
steps = [make(i) for i in range(6)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for run, _ in steps:
        run()
for _ in range(2):
    for _, out in steps:
        wipe(out)
    graph.replay()
torch.cuda.synchronize()
got = [{n: t.clone() for n, t in out.items()} for _, out in steps]
for (run, out), g in zip(steps, got):
    wipe(out)
    run()
    torch.cuda.synchronize()
    for n, t in out.items():
        assert torch.equal(t.view(torch.uint8), g[n].view(torch.uint8)), n
assert qg.qg_device_error() == 0
print("OK")
'''

THREADS = r'''
import threading
steps = [make(i) for i in range(6)]
torch.cuda.synchronize()
errors = []
def work(i):
    try:
        run, out = steps[i]
        s = torch.cuda.Stream()
        for _ in range(20):
            run(stream=s)
        s.synchronize()
    except Exception as e:
        errors.append(repr(e))
threads = [threading.Thread(target=work, args=(i,)) for i in range(6)]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert not errors, errors
got = [{n: t.clone() for n, t in out.items()} for _, out in steps]
for (run, out), g in zip(steps, got):
    wipe(out)
    run()
    torch.cuda.synchronize()
    for n, t in out.items():
        assert torch.equal(t.view(torch.uint8), g[n].view(torch.uint8)), n
assert qg.qg_device_error() == 0
print("OK")
'''


@pytest.mark.parametrize("code", [CAPTURE, THREADS], ids=["capture", "threads"])
def test_fresh_process(code):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", "ROOT = " + repr(ROOT) + "\n" + COMMON + code], cwd=ROOT,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-3000:])
    assert "OK" in r.stdout
