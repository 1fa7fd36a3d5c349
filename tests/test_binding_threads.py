"""First calls of the binding from several host threads. What it looks up on first use is checked at every bytecode boundary
of the look-up: there another thread makes its own first call, which must come out right. No GPU needed."""
import sys
import threading

import pytest

import gemm_q4_q8_gb300 as qg
from gemm_q4_q8_gb300 import build as qbuild

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qbuild.build()
    qg.load()


def interrupted(code, first, other):
    """first(), with other() run to its end in another thread before each bytecode of `code`; how often that was."""
    fails, count = [], [0]

    def thread():
        try:
            other()
        except Exception as e:
            fails.append(repr(e))

    def trace(frame, event, arg):
        if frame.f_code is not code:
            return None
        frame.f_trace_opcodes = True
        if event == "opcode":
            count[0] += 1
            t = threading.Thread(target=thread)
            t.start()
            t.join()
        return trace
    was = sys.gettrace()
    sys._getframe().f_trace_opcodes = True  # (3.12 looks for one such frame when tracing starts)
    sys.settrace(trace)
    try:
        first()
    finally:
        sys.settrace(was)
    assert not fails, fails[0]
    return count[0]


def test_current_stream(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    names = ("_raw_stream", "_device")

    def other():
        was = {n: getattr(qg, n) for n in names}
        assert qg._stream(None) == 1003
        for n, v in was.items():  # the other thread's own look-up is taken back: every boundary is its first call
            setattr(qg, n, v)
    for n in names:
        monkeypatch.setattr(qg, n, None)
    assert interrupted(qg._stream.__code__, lambda: qg._stream(None), other) > 10
    assert qg._stream(None) == 1003


def test_element_types(monkeypatch):
    names = ("_ELEM", "_INT32", "_FLOAT16")
    for n in names:
        monkeypatch.setattr(qg, n, None)
    table, pool = torch.zeros((1, 1), dtype=torch.int32), torch.zeros(qg.qkv_page_bytes(8, 2, 64, 16), dtype=torch.uint8)
    cache = qg.QGKVCache(pool.data_ptr(), table.data_ptr(), 8, 2, 64, 16, 1, 1, 1)
    k, pos = torch.zeros(0, 2, 64), torch.zeros(0, dtype=torch.int32)
    q, q_out = torch.zeros(0, 4, 64), torch.zeros(0, 4, 64, dtype=torch.float16)
    one = torch.zeros(1, 1, 4, 64, dtype=torch.float16)

    def calls():  # none of them gets as far as a device: no tokens, no workspace
        was = {n: getattr(qg, n) for n in names}
        qg.qkv_append(cache, k, k, pos, q=q, q_out=q_out, stream=0)
        for n, v in was.items():
            setattr(qg, n, v)
        with pytest.raises(qg.QGError) as e:
            qg.qattn_paged(cache, one, torch.zeros(1, dtype=torch.int32), torch.zeros_like(one), pool[:0], stream=0)
        assert e.value.status == qg.QG_ERR_WORKSPACE
        for n, v in was.items():
            setattr(qg, n, v)
    assert interrupted(qg._dtypes.__code__, lambda: qg._elem(k, "k"), calls) > 10
    calls()
