"""The dense gated block where its products run on CTA pairs (tiles of 256 x 256, with and without a split of the
depth), its deep sums, and few tokens on wide blocks.  Bounds: tests/dense_util.py."""
import pytest
import torch

import expert_offloaded_edge_b200 as ftm
from tests import dense_util as du
from tests.test_gpu_gated_ffn import CANARY, Block, normal

pytestmark = pytest.mark.gpu

# A product leaves the few-token engine above 74 tiles of 128 tokens x 128 outputs (64 for gate/up), 148 up to 2048
# deep, and its pairs' tile is split along the depth up to 37 tiles and from 512 deep.
GATED_SPLIT = [(1500, 2176, 512), (1270, 2176, 512)]       # gate/up: 24 tiles on two pairs each, 20 on three
DGATE_SPLIT = [(1500, 2176, 1024), (1270, 2176, 1024)]     # activation gradient split, gate/up on pairs
DOWN_SPLIT = [(1500, 1024, 2176), (1270, 1024, 2176)]      # down split, gate/up and activation gradient on pairs
WHOLE = [(4100, 256, 1280), (9000, 384, 640)]              # gate/up and activation gradient on pairs, several tiles to each
PAIRS = GATED_SPLIT + DGATE_SPLIT + DOWN_SPLIT + WHOLE
ONE_EACH = [GATED_SPLIT[1], DGATE_SPLIT[1], DOWN_SPLIT[0], WHOLE[0]]


@pytest.mark.parametrize("T,d,I", PAIRS)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_block_and_gradients_on_pairs(T, d, I, act):
    b = Block(T, d, I, act, seed=T + I)
    b.forward(pre=False)
    b.done()
    b.check_forward(pre=False)
    bare = b.y.clone()
    outs = []
    for _ in range(2):
        b.ws.fill_(255)                  # stale workspaces are never read (0xffff is a NaN)
        b.forward()
        b.backward()
        b.done()
        outs.append([t.clone() for t in (b.y, b.pre, b.dx, b.dbank)])
    b.check_forward()
    b.check_backward()
    assert torch.equal(b.y, bare)
    assert all(torch.equal(p, q) for p, q in zip(*outs))


@pytest.mark.parametrize("T,d,I", ONE_EACH)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_one_of_the_gradients_on_pairs(T, d, I, act):
    b = Block(T, d, I, act, seed=3)
    b.forward()
    b.backward()
    b.done()
    both = b.dx.clone(), b.dbank.clone()
    for dx, dbank in ((True, False), (False, True)):
        b.dx.fill_(CANARY)
        b.dbank.fill_(CANARY)
        b.backward(dx, dbank)
        b.done()
        b.check_backward(dx, dbank)
        assert torch.equal(b.dx if dx else b.dbank, both[0] if dx else both[1])


@pytest.mark.parametrize("T,d,I", ONE_EACH)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_a_broken_row_stays_in_its_row_on_pairs(T, d, I, act):
    b = Block(T, d, I, act)
    b.forward()
    b.backward()
    b.done()
    y, pre, dx = b.y.clone(), b.pre.clone(), b.dx.clone()
    bad = T // 2
    b.x[bad, 3], b.x[bad, 17] = float("nan"), float("inf")
    b.dy[bad] = float("nan")
    b.forward()
    b.backward(dbank=False)
    b.done()
    keep = torch.arange(T + 1, device="cuda") != bad
    assert torch.equal(b.y[keep], y[keep]) and torch.equal(b.pre[keep], pre[keep]) and torch.equal(b.dx[keep], dx[keep])
    assert bool(b.y[bad].isnan().all()) and bool(b.dx[bad].isnan().all())


@pytest.mark.parametrize("T,d,I", ONE_EACH)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_a_nan_that_was_kept_reaches_the_gradients_on_pairs(T, d, I, act):
    b = Block(T, d, I, act, seed=23)
    b.forward()
    b.pre[T // 2, 77] = float("nan")
    b.backward()
    b.done()
    n = 2 * I * d
    dwg = b.dbank[:n // 2].view(I, d).isnan()
    assert bool(dwg[77].all()) and int(dwg.sum()) == d
    dwd = b.dbank[n:n + n // 2].view(d, I).isnan()
    assert bool(dwd[:, 77].all()) and int(dwd.sum()) == d
    dx = b.dx[:T].isnan()
    assert bool(dx[T // 2].all()) and int(dx.sum()) == d


@pytest.mark.parametrize("T,d,I", ONE_EACH)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_far_values_of_the_activation_on_pairs(T, d, I, act):
    """Planted g and u far outside of the activation's curved part: slopes 0 and 1, never NaN."""
    b = Block(T, d, I, act)
    far = torch.tensor([-1e38, -3e19, -1e6, -200.0, -90.0, 90.0, 200.0, 1e6, 3e19, 1e38], device="cuda")
    b.pre[:T, :I] = far[torch.arange(T * I, device="cuda") % far.numel()].view(T, I).to(torch.bfloat16)
    b.pre[:T, I:] = 0.5
    b.dy.mul_(1e-3)
    b.bank[2 * I * d:].mul_(1e-3)
    b.backward(dbank=False)
    b.done()
    # at +-90 sigmoid is 0 or 1 to 90 e^-90: dg = dh u and du = dh g on the right, 0 on the left
    g, u = b.pre[:T, :I].double(), 0.5
    _, _, wd = du.split_bank(b.bank, d, I)
    dh = b.dy.double() @ wd
    e = du.gamma(d) * (b.dy.double().abs() @ wd.abs())
    on = (g > 0).double()
    dgu, e_dgu = torch.cat([on * dh * u, on * dh * g], 1), torch.cat([on * e * u, on * e * g], 1)
    e_dgu = e_dgu + du.U * (dgu.abs() + e_dgu) + du.FAST * dgu.abs()
    w = torch.cat(du.split_bank(b.bank, d, I)[:2])
    want = dgu @ w
    bound = e_dgu @ w.abs() + du.gamma(2 * I) * ((dgu.abs() + e_dgu) @ w.abs())
    du.assert_within(b.dx[:T], want, bound + du.U * (want.abs() + bound), "dx")


@pytest.mark.parametrize("T,d,I", ONE_EACH)
def test_captured_and_on_two_streams_on_pairs(T, d, I):
    b, c = Block(T, d, I, "gelu", seed=1), Block(T - 77, d, I, "silu", seed=2)
    b.forward()
    b.backward()
    b.done()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        b.forward()
        b.backward()
    for seed in (50, 60):
        b.x.copy_(normal(seed, T, d))
        b.dy.copy_(normal(seed + 1, T, d))
        graph.replay()
        b.done()
        b.check_forward()
        b.check_backward()
    want = [t.clone() for t in (b.y, b.dx, b.dbank)]
    streams = (torch.cuda.Stream(), torch.cuda.Stream())
    torch.cuda.synchronize()
    for _ in range(5):
        for k, s in zip((b, c), streams):
            k.forward(stream=s)
            k.backward(stream=s)
    b.done()
    assert all(torch.equal(p, q) for p, q in zip((b.y, b.dx, b.dbank), want))
    c.check_forward()
    c.check_backward()


# a few tokens on a block so wide that gate/up leaves the few-token engine
@pytest.mark.parametrize("T,d,I", [(9, 2176, 5120), (32, 2176, 5120), (64, 256, 9600), (128, 256, 9600), (17, 9728, 256)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_few_tokens_on_wide_blocks(T, d, I, act):
    b = Block(T, d, I, act, seed=T)
    b.forward()
    b.backward()
    b.done()
    b.check_forward()
    b.check_backward()


@pytest.mark.parametrize("T,d,I", [(20000, 256, 128), (12983, 768, 128), (9000, 384, 640), (4100, 256, 1280), (100000, 128, 128)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_deep_sums_leave_nothing_out(T, d, I, act):
    """The worst case's bounds grow with the depth until a block of 64 tokens left out would pass them; the error's
    norm does not (tests/test_dense_abi.py shows what it sees)."""
    b = Block(T, d, I, act, seed=T)
    b.forward()
    b.backward()
    b.done()
    (dx, dw, dwd), _ = du.block_backward(b.x, b.bank, b.pre[:T], b.dy, d, I, act)
    n = 2 * I * d
    assert du.norm_error(b.dbank[:n].view(2 * I, d), dw) <= du.NORM
    assert du.norm_error(b.dbank[n:3 * I * d].view(d, I), dwd) <= du.NORM
    assert du.norm_error(b.dx[:T], dx) <= du.NORM
