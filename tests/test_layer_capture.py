"""The norm, the lookup, the routing and the 4-bit cache's calls made for the first time inside CUDA-graph capture, in a fresh
process, and from several host threads at once: every output equals the eager call's, bit for bit."""
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
    """A step of its own sizes and types: (run, outputs)."""
    kv, heads, d, ps, ncols, lens = ((8, 40, 128, 64, 1, [700, 5000, 1]), (2, 16, 256, 16, 1, [1000]), (4, 32, 64, 32, 8, [2000, 3, 800, 0]),
                                     (1, 17, 64, 16, 16, [300, 17]), (2, 16, 256, 128, 4, [900, 1234]), (8, 8, 128, 256, 3, [50] * 30))[i]
    hidden, rows, experts, k, src, dst = ((5120, 33, 256, 8, 0, 0), (2048, 1, 64, 4, 1, 0), (96, 700, 40, 3, 0, 1), (8192, 5, 512, 10, 1, 1),
                                          (32, 3000, 1024, 32, 0, 2), (1056, 200, 16, 2, 1, 2))[i]
    table = (qg.Q4_0, qg.Q8_0, qg.QG_F16)[i % 3]
    n = len(lens)
    pages = -(-max(lens) // ps) + 1
    g = torch.Generator(device="cuda").manual_seed(i)
    pool = torch.full((n * pages * qg.qkv_page_bytes(qg.Q4_1, kv, d, ps),), 0xFF, dtype=torch.uint8, device="cuda")
    place = torch.randperm(n * pages, generator=g, device="cuda").to(torch.int32).view(n, pages)
    c = qg.qkv_cache(qg.Q4_1, pool, place, kv, d, ps)
    plan = qg.qrope_plan(d // 2, interleaved=bool(i % 2))
    pos = torch.tensor([j for m in lens for j in range(m)], dtype=torch.int32, device="cuda")
    seq = torch.tensor([s for s, m in enumerate(lens) for _ in range(m)], dtype=torch.int32, device="cuda")
    qkv = torch.randn(len(pos), heads + 2 * kv, d, generator=g, device="cuda")
    last = torch.tensor([max(m - ncols, 0) + t for m in lens for t in range(ncols)], dtype=torch.int32, device="cuda")
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(qg.qattn_workspace_bytes(c, heads, ncols), dtype=torch.uint8, device="cuda")
    queries = torch.randn(n, ncols, heads, d, generator=g, device="cuda").half()
    kind = (torch.float32, torch.float16)[src]
    x, add = (torch.randn(rows, hidden, generator=g, device="cuda").to(kind) for _ in range(2))
    w = torch.rand(hidden, generator=g, device="cuda") + 0.5
    if table == qg.QG_F16:
        q, scl = torch.randn(100, hidden, generator=g, device="cuda").half(), None
    else:
        q = torch.randint(0, 256, (100, hidden if table == qg.Q8_0 else hidden // 2), generator=g, device="cuda", dtype=torch.uint8)
        scl = (torch.rand(100, hidden // 32, generator=g, device="cuda") * 0.01).half()
    ids = torch.randint(0, 100, (rows,), generator=g, device="cuda").to(torch.int32)
    wr = torch.randn(experts, hidden, generator=g, device="cuda") * hidden ** -0.5
    bias = torch.randn(experts, generator=g, device="cuda") * 0.1 if i % 2 else None
    route = qg.qroute_plan(("softmax", "sigmoid")[i % 2], n_group=4, top_group=2 + i % 2, group_top=1 + i % 2)
    logits = torch.randn(rows, experts, generator=g, device="cuda")
    cols = min(rows, 16)
    xs = torch.randn(cols, hidden, generator=g, device="cuda").half()
    f = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda")
    out = dict(q=f(len(pos), heads, d, dtype=torch.float16), k=f(n * ncols, kv, d, dtype=torch.float16), v=f(n * ncols, kv, d, dtype=torch.float16),
               y=f(n, ncols, heads, d, dtype=torch.float16), pool=pool, s=f(rows, hidden, dtype=kind), e=f(rows, hidden, dtype=kind),
               ids=f(rows, k, dtype=torch.int32), rw=f(rows, k), ids2=f(cols, k, dtype=torch.int32), rw2=f(cols, k), lg=f(cols, experts))
    if dst == 2:
        out.update(n=f(rows, hidden, dtype=torch.int8), ns=f(rows, hidden // 32, dtype=torch.float16))
    else:
        out.update(n=f(rows, hidden, dtype=(torch.float32, torch.float16)[dst]))
    def run(stream=None):
        qg.qkv_append(c, qkv[:, heads:heads + kv], qkv[:, heads + kv:], pos, seq=seq, rope=plan, q=qkv[:, :heads], q_out=out["q"], stream=stream)
        qg.qkv_read(c, last, out["k"], out["v"], stream=stream)
        qg.qattn_paged(c, queries, lens_d, out["y"], ws, stream=stream)
        qg.qrms_norm(x, w, out["n"], add=add, sum_out=out["s"], y_scl=out.get("ns"), stream=stream)
        qg.qembed(table, q, scl, ids, out["e"], scale=1.5, stream=stream)
        qg.qmoe_route(route, logits, k, out["ids"], out["rw"], bias=bias, stream=stream)
        qg.qmoe_router_planned(route, wr, xs, k, out["ids2"], out["rw2"], bias=bias, logits_out=out["lg"], stream=stream)
    return run, out

def wipe(out):
    for n, t in out.items():
        t.fill_(0xFF if n == "pool" else 7)

def same(steps, got):
    for (run, out), g in zip(steps, got):
        wipe(out)
        run()
        torch.cuda.synchronize()
        for n, t in out.items():
            assert torch.equal(t.view(torch.uint8), g[n].view(torch.uint8)), n
    assert qg.qg_device_error() == 0
    print("OK")
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
same(steps, [{n: t.clone() for n, t in out.items()} for _, out in steps])
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
same(steps, [{n: t.clone() for n, t in out.items()} for _, out in steps])
'''


@pytest.mark.parametrize("code", [CAPTURE, THREADS], ids=["capture", "threads"])
def test_fresh_process(code):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", "ROOT = " + repr(ROOT) + "\n" + COMMON + code], cwd=ROOT, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-3000:])
    assert "OK" in r.stdout
