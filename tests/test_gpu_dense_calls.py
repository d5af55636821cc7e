"""The dense operators called as programs call them: inputs written just before, the first call of a process captured,
several host threads at once, memory of torch's expandable segments."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import expert_offloaded_edge_b200 as ftm
from tests.test_gpu_gated_ffn import Block, normal
from tests.test_gpu_lora import Linear, adapters_of

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("T,d,I", [(1, 512, 384), (12, 256, 640), (40, 512, 384), (200, 384, 256), (1270, 2176, 512), (9000, 384, 640)])
def test_the_block_reads_what_was_written_just_before(T, d, I):
    """Weights, x and dy change in the same stream before every call; launches that start early never see the old ones."""
    b = Block(T, d, I)
    sets = [(normal(s, T, d), normal(s + 1, 3 * I * d, std=0.05), normal(s + 2, T, d)) for s in (60, 70, 80)]
    outs = (b.y, b.pre, b.dx, b.dbank)

    def call(k):
        for to, src in zip((b.x, b.bank, b.dy), sets[k]):
            to.copy_(src)
        b.forward()
        b.backward()
        return [t.clone() for t in outs]

    want = []
    for k in range(3):
        want.append(call(k))
        b.done()
        b.check_forward()
        b.check_backward()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(150):
        for p, q in zip(call(i % 3), want[i % 3]):
            wrong += (p != q).any()
    b.done()
    assert int(wrong) == 0


@pytest.mark.parametrize("T,d_in,d_out,rank", [(3, 512, 384, 16), (12, 520, 384, 24), (200, 512, 640, 16), (640, 520, 2048, 40),
                                               (2500, 264, 2048, 16)])
def test_the_projection_reads_what_was_written_just_before(T, d_in, d_out, rank):
    m = Linear(T, d_in, d_out, 5, rank, "mixed")
    sets = [(normal(s, T, d_in), normal(s + 1, d_out, d_in, std=0.1), normal(s + 2, 5, rank, d_in, std=0.1),
             normal(s + 3, 5, d_out, rank, std=0.3), adapters_of(T, 5, mix, s)) for s, mix in ((60, "mixed"), (70, "distinct"), (80, "runs"))]

    def call(k):
        for to, src in zip((m.x, m.w, m.a, m.b, m.ids), sets[k]):
            to.copy_(src)
        m.run()
        return m.y.clone()

    want = []
    for k in range(3):
        want.append(call(k))
        m.done()
        m.check()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(150):
        wrong += (call(i % 3) != want[i % 3]).any()
    m.done()
    assert int(wrong) == 0


CHILD = """
import torch
from tests.test_gpu_gated_ffn import Block
from tests.test_gpu_lora import Linear
blocks = [Block(T, d, I, act) for T, d, I, act in ((4, 256, 128, "silu"), (40, 256, 128, "gelu"), (1270, 2176, 512, "silu"), (5000, 256, 128, "gelu"))]
linears = [Linear(T, 512, do, 5, 16, "mixed") for T, do in ((3, 256), (40, 256), (640, 2048), (2500, 2048))]
torch.cuda.synchronize()
def calls():
    for b in blocks:
        b.forward()
        b.backward()
    for m in linears:
        m.run()
{body}
for b in blocks:
    b.done()
    b.check_forward()
    b.check_backward()
for m in linears:
    m.done()
    m.check()
print("child done")
"""


@pytest.mark.parametrize("body,env", [
    ("g = torch.cuda.CUDAGraph()\nwith torch.cuda.graph(g):\n    calls()\ng.replay()", {}),       # nothing of the library ran before
    ("calls()", {"PYTORCH_CUDA_ALLOC_CONF": "expandable_segments:True"})])
def test_first_calls_of_a_process(body, env):
    p = subprocess.run([sys.executable, "-c", CHILD.replace("{body}", body)], cwd=ROOT, env={**os.environ, **env},
                       capture_output=True, text=True, timeout=240)
    assert p.returncode == 0 and "child done" in p.stdout, p.stdout[-2000:] + p.stderr[-2000:]


def in_a_new_thread(f):
    errors = []

    def run():
        try:
            f()
        except BaseException as e:      # noqa: BLE001 (raised again below)
            errors.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("T", [5, 60, 1500, 5000])
def test_the_first_call_of_a_host_thread(T):
    """A thread that has made no CUDA call of its own has no current context yet: each call gives it one."""
    L, i32 = ftm.LayerDesc(512, 16, 2, 384, 0, 16, ftm.FTM_BF16, 0), dict(dtype=torch.int32, device="cuda")
    b, m, stream = Block(T, 512, 384), Linear(T, 512, 2048, 6, 32), torch.cuda.current_stream().cuda_stream
    wr, ids, gates = normal(5, 16, 512), torch.full((2, T, 2), -1, **i32), torch.zeros(2, T, 2, device="cuda")
    ftm.ftm_route(L, b.x, T, wr, None, ids[0], gates[0])
    torch.cuda.synchronize()
    for call in (lambda: b.forward(stream=stream), lambda: b.backward(stream=stream), lambda: m.run(stream),
                 lambda: ftm.ftm_route(L, b.x, T, wr, None, ids[1], gates[1], stream)):
        in_a_new_thread(call)
    b.done()
    b.check_forward()
    b.check_backward()
    m.check()
    assert torch.equal(ids[0], ids[1]) and torch.equal(gates[0], gates[1])


def test_host_threads_at_once():
    work = [Block(T, 512, 384, act, seed=T) for T, act in ((5, "silu"), (60, "gelu"), (1500, "silu"))]
    work += [Linear(T, 512, 2048, 6, 32, mix, seed=T) for T, mix in ((3, "distinct"), (90, "mixed"), (1200, "runs"))]
    errors = []

    def loop(w):
        try:
            s = torch.cuda.Stream()
            for _ in range(30):
                if isinstance(w, Block):
                    w.forward(stream=s)
                    w.backward(stream=s)
                else:
                    w.run(s)
                with pytest.raises(ftm.FtmError, match="workspace"):     # each thread keeps its own last error
                    ftm.ftm_gated_ffn(ftm.LayerDesc(256, 1, 1, 128, 0, 1, ftm.FTM_BF16, 0), 0, w.x, 4, w.x, None, w.x, None, 0, s)
            s.synchronize()
        except BaseException as e:      # noqa: BLE001 (reported by the main thread)
            errors.append(repr(e))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=loop, args=(w,)) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    assert ftm.ftm_device_status(True) == 0
    for w in work:
        if isinstance(w, Block):
            w.check_forward()
            w.check_backward()
        else:
            w.check()


@pytest.mark.parametrize("T,d,I", [(1, 2048, 768), (8, 512, 256), (12, 2048, 128), (40, 512, 256)])
@pytest.mark.parametrize("graph", [False, True])
def test_weights_that_the_launch_before_wrote(T, d, I, graph):
    """The down weights are the output of an adapter projection right in front of the block, so that between their
    writing and the down launch, which reads them early, there are only launches that start early themselves."""
    b, n = Block(T, d, I), 8
    w_d = b.bank[2 * I * d:].view(d, I)
    m = Linear(d, 128, I, 2, 8, "none", std=0.1)
    xs = [normal(10 + i, d, 128, std=0.05) for i in range(n)]
    ys = torch.zeros(n, T, d, dtype=torch.bfloat16, device="cuda")

    def chain():
        for i in range(n):
            ftm.ftm_lora_linear(m.D, xs[i], d, m.w, m.a, m.b, None, m.ids, w_d, m.ws, m.ws.numel())
            b.forward(pre=False, y=ys[i])

    want = []
    for i in range(n):
        ftm.ftm_lora_linear(m.D, xs[i], d, m.w, m.a, m.b, None, m.ids, w_d, m.ws, m.ws.numel())
        torch.cuda.synchronize()
        b.forward(pre=False)
        b.done()
        b.check_forward(pre=False)
        want.append(b.y[:T].clone())
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            chain()
        call = g.replay
    else:
        call = chain
    for _ in range(30):
        ys.zero_()
        call()
        b.done()
        assert torch.equal(ys, torch.stack(want))


@pytest.mark.parametrize("T,d,I", [(3, 1 << 20, 128), (40, 1 << 20, 128), (3, 128, 1 << 20), (40, 128, 1 << 20)])
def test_the_block_at_the_largest_widths(T, d, I):
    b = Block(T, d, I, "silu", seed=T)
    b.bank.mul_(0.1)
    b.forward()
    b.backward()
    b.done()
    b.check_forward()
    b.check_backward()


@pytest.mark.parametrize("T,d_in,d_out,n,rank", [(2, 1 << 20, 64, 2, 8), (40, 1 << 20, 64, 2, 24), (2, 64, 1 << 20, 2, 8),
                                                 (40, 64, 1 << 20, 3, 16), (70, 64, 128, 65536, 8), (3, 64, 128, 65536, 8)])
def test_adapters_at_the_largest_sizes(T, d_in, d_out, n, rank):
    m = Linear(T, d_in, d_out, n, rank, "distinct", seed=T)
    m.ids[0] = n - 1
    m.run()
    m.done()
    m.check()
