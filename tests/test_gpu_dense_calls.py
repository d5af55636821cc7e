"""The dense operators called as programs call them: from new host threads, several of
them at once."""
import threading

import pytest
import torch

import expert_offloaded_edge_b200 as ftm
from tests.test_gpu_gated_ffn import Block, normal
from tests.test_gpu_lora import Linear

pytestmark = pytest.mark.gpu


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
