"""The shared projection with adapters of many requests on the GPU, against a 64-bit reference with bounds that
follow from the arithmetic (tests/dense_util.py)."""
import pytest
import torch

import expert_offloaded_edge_b200 as ftm
from tests import dense_util as du

pytestmark = pytest.mark.gpu

CANARY = 7.0


def normal(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def adapters_of(T, n, mix, seed=0):
    """Adapter ids of T tokens: one for all, none, runs (packed prompts), mixed per token, or runs that come back."""
    g = torch.Generator().manual_seed(seed)
    if mix == "one":
        ids = torch.full((T,), n - 1)
    elif mix == "none":
        ids = torch.full((T,), -1)
    elif mix == "mixed":
        ids = torch.randint(-1, n, (T,), generator=g)
    elif mix == "distinct":
        ids = torch.randperm(max(n, T), generator=g)[:T] % n
    else:
        lengths = max(1, T // 7)
        ids = (torch.arange(T) // lengths) % (n + 1) - 1
    return ids.to(torch.int32).cuda()


class Linear:
    def __init__(self, T, d_in, d_out, n, rank, mix="mixed", seed=0, scaled=True, std=0.3):
        self.D = ftm.LoraDesc(d_in, d_out, n, rank, ftm.FTM_BF16, 0)
        self.T = T
        self.x, self.w = normal(seed, T, d_in), normal(seed + 1, d_out, d_in, std=0.1)
        self.a, self.b = normal(seed + 2, n, rank, d_in, std=0.1), normal(seed + 3, n, d_out, rank, std=std)
        g = torch.Generator(device="cuda").manual_seed(seed + 4)
        self.scale = (torch.rand(n, generator=g, device="cuda") * 2 - 0.5) if scaled else None
        self.ids = adapters_of(T, n, mix, seed)
        self.y = torch.full((T + 1, d_out), CANARY, dtype=torch.bfloat16, device="cuda")
        self.ws = torch.empty(max(256, ftm.ftm_lora_workspace_bytes(self.D, T)), dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        ftm.ftm_lora_linear(self.D, self.x, self.T, self.w, self.a, self.b, self.scale, self.ids, self.y, self.ws,
                            self.ws.numel(), stream)

    def done(self, status=0):
        torch.cuda.synchronize()
        assert ftm.ftm_device_status(True) == status

    def check(self):
        want, bound = du.lora(self.x, self.w, self.a, self.b, self.scale, self.ids)
        du.assert_within(self.y[:self.T], want, bound, "y")
        assert bool((self.y[self.T:] == CANARY).all())


@pytest.mark.parametrize("T,d_in,d_out,n,rank,mix", [
    # one tile of few tokens, every token tile width, odd sizes, ranks that pad to 16, K and outputs below a block
    (1, 8, 8, 1, 8, "one"), (1, 2048, 512, 3, 16, "one"), (2, 72, 24, 2, 8, "mixed"), (5, 200, 136, 4, 24, "distinct"),
    (16, 256, 128, 16, 16, "distinct"), (17, 256, 264, 4, 40, "mixed"), (33, 1000, 128, 7, 64, "mixed"),
    (64, 512, 1736, 64, 16, "distinct"), (65, 128, 384, 9, 128, "mixed"), (77, 1000, 136, 5, 24, "runs"),
    (128, 320, 1000, 128, 8, "distinct"), (130, 136, 72, 3, 8, "none"), (200, 264, 392, 17, 96, "mixed"),
    # CTA pairs: one tile and many to a pair, tiles without adapters, all adapters in every tile (a tile split along K: SPLIT_PAIRS)
    (300, 1024, 8200, 5, 32, "runs"), (512, 520, 4104, 33, 16, "mixed"), (513, 256, 6152, 4, 48, "runs"),
    (700, 64, 4096, 700, 8, "distinct"), (1100, 1024, 4096, 6, 80, "runs"), (1030, 200, 7000, 3, 112, "one"),
    (2500, 328, 2056, 9, 32, "runs"), (2600, 128, 4096, 12, 64, "mixed"), (5000, 64, 2048, 40, 16, "runs"),
    (4100, 8, 2048, 2, 128, "none")])
def test_projection(T, d_in, d_out, n, rank, mix):
    m = Linear(T, d_in, d_out, n, rank, mix, seed=T)
    m.run()
    m.done()
    m.check()


@pytest.mark.parametrize("T,d_in,d_out,n,rank,mix", [
    # a handful of tokens: one launch up to 8 tokens and 8 groups of 16 adapter rows, in clusters of 4 or 8; beyond, two
    (1, 24, 40, 2, 128, "one"), (1, 6144, 264, 3, 72, "one"), (3, 8, 136, 3, 16, "none"), (4, 4096, 1000, 9, 16, "distinct"),
    (4, 200, 520, 9, 32, "distinct"), (4, 72, 128, 9, 40, "distinct"), (5, 1032, 16, 5, 8, "distinct"),
    (7, 328, 248, 3, 16, "mixed"), (8, 136, 72, 8, 16, "distinct"), (8, 512, 2056, 12, 8, "distinct"),
    (8, 512, 72, 12, 24, "distinct"), (9, 512, 72, 12, 8, "distinct"), (2, 64, 4544, 2, 24, "mixed"),
    (2, 1024, 4552, 2, 64, "distinct"), (2, 1032, 4552, 2, 64, "distinct"), (6, 264, 8456, 6, 16, "distinct"),
    (3, 64, 9096, 3, 16, "distinct"), (8, 40, 128, 1, 16, "one")])
@pytest.mark.parametrize("scaled", [True, False])
def test_a_handful_of_tokens(T, d_in, d_out, n, rank, mix, scaled):
    m = Linear(T, d_in, d_out, n, rank, mix, seed=T + rank, scaled=scaled)
    m.run()
    m.done()
    m.check()


def test_a_handful_of_tokens_between_two_streams_and_in_a_graph():
    """Clusters of 4 and 8 in turn, in one graph and on two streams at once."""
    a, b = Linear(3, 2048, 2048, 5, 16, "distinct", seed=1), Linear(8, 1000, 4104, 8, 16, "distinct", seed=2)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for m, st in zip((a, b), streams):
            m.run(st)
    a.done()
    a.check()
    b.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for m in (a, b, a, b):
            m.run()
    for m in (a, b):
        m.x.copy_(normal(9, *m.x.shape))
        m.ids.copy_(adapters_of(m.T, m.D.n_adapters, "mixed", 4))
        m.y.fill_(CANARY)
    g.replay()
    a.done()
    a.check()
    b.check()


def test_a_handful_of_tokens_is_isolated_and_strided():
    T, d_in, d_out = 8, 264, 200
    m = Linear(T, d_in, d_out, 8, 16, "distinct", seed=3)
    m.ids[1], m.ids[5] = m.ids[0], -1
    big = torch.full((T + 2, d_in + d_out + 48), CANARY, dtype=torch.bfloat16, device="cuda")
    x, y = big[:T, 16:16 + d_in], big[:T, d_in + 32:d_in + 32 + d_out]
    x.copy_(m.x)
    before = big.clone()

    def run():
        ftm.ftm_lora_linear(m.D, x, T, m.w, m.a, m.b, m.scale, m.ids, y, m.ws, m.ws.numel(), ldx=big.stride(0),
                            ldy=big.stride(0))
        m.done()
    run()
    want, bound = du.lora(m.x, m.w, m.a, m.b, m.scale, m.ids)
    du.assert_within(y, want, bound, "y")
    before[:T, d_in + 32:d_in + 32 + d_out] = y
    assert torch.equal(big, before)
    clean = y.clone()
    a2, a3, a4 = (int(m.ids[t]) for t in (2, 3, 4))
    m.a[a2, 3, 7], m.b[a3, ::5, 2], m.scale[a4] = float("nan"), float("inf"), float("nan")
    x[6, 1] = float("inf")
    run()
    broken = torch.tensor([t in (2, 3, 4, 6) for t in range(T)], device="cuda")
    broken |= torch.isin(m.ids, m.ids[torch.tensor([2, 3, 4], device="cuda")])
    assert torch.equal(y[~broken], clean[~broken])
    assert bool(y[2].isnan().all()) and bool(y[4].isnan().all()) and not bool(torch.isfinite(y[6]).any())
    assert not bool(torch.isfinite(y[3, ::5]).any())
    own = torch.arange(d_out, device="cuda") % 5 != 0
    assert torch.equal(y[3, own], clean[3, own])


@pytest.mark.parametrize("T", [12, 600])
def test_without_scales(T):
    m = Linear(T, 256, 4096, 5, 16, scaled=False)
    m.run()
    m.done()
    m.check()


@pytest.mark.parametrize("T", [1, 60, 500, 2100])
def test_ids_out_of_range_take_no_adapter_and_are_reported(T):
    m = Linear(T, 256, 2048, 4, 16, "runs")
    m.ids[::3] = 4
    m.ids[T // 2] = -2
    m.ids[T - 1] = 2 ** 31 - 1
    m.run()
    m.done(status=2)
    m.check()
    m.run()
    torch.cuda.synchronize()
    assert ftm.ftm_device_status(True) == 2


@pytest.mark.parametrize("T", [50, 500, 2500])
def test_a_reported_id_stops_no_later_call(T):
    """The status word keeps a reported id until it is read; calls in between compute all the same (their waits
    do not take it for a wait that gave up)."""
    bad = Linear(4, 256, 128, 2, 16)
    bad.ids[0] = 9
    bad.run()
    m = Linear(T, 4096, 4096, 8, 32, "mixed", seed=T)
    for _ in range(5):
        m.run()
    m.done(status=2)
    m.check()


@pytest.mark.parametrize("T,d_out", [(40, 200), (300, 8200), (2500, 2048)])
def test_slices_of_one_matrix(T, d_out):
    """x and y are column slices of one matrix; the columns around them and the rows behind stay as they were."""
    d_in = 264
    m = Linear(T, d_in, d_out, 6, 24, "runs", seed=3)
    big = torch.full((T + 2, d_in + d_out + 48), CANARY, dtype=torch.bfloat16, device="cuda")
    x, y = big[:T, 16:16 + d_in], big[:T, d_in + 32:d_in + 32 + d_out]
    x.copy_(m.x)
    before = big.clone()
    ftm.ftm_lora_linear(m.D, x, T, m.w, m.a, m.b, m.scale, m.ids, y, m.ws, m.ws.numel(), ldx=big.stride(0),
                        ldy=big.stride(0))
    m.done()
    want, bound = du.lora(m.x, m.w, m.a, m.b, m.scale, m.ids)
    du.assert_within(y, want, bound, "y")
    before[:T, d_in + 32:d_in + 32 + d_out] = y
    assert torch.equal(big, before)


@pytest.mark.parametrize("T,d_out,mix", [(24, 256, "mixed"), (100, 4096, "mixed"), (600, 6152, "runs"), (2500, 2048, "mixed")])
def test_requests_are_isolated(T, d_out, mix):
    """What another request's row or adapter holds does not change a bit of a token's result: infinities and NaN in
    one adapter's A, B and scale and in another's tokens."""
    m = Linear(T, 320, d_out, 6, 40, mix, seed=11)
    m.run()
    m.done()
    clean = m.y.clone()
    m.a[0, 3, 7], m.a[0, 5, 9] = float("nan"), float("inf")
    m.b[1, ::5, 2] = float("inf")
    m.b[1, 1::5, 39] = float("nan")
    m.b[1, 2, 8] = -float("inf")
    m.scale[2] = float("nan")
    rows = torch.arange(T, device="cuda")
    broken = (m.ids == 3) & (rows % 2 == 0)
    m.x[broken, 1] = float("inf")
    m.run()
    m.done()
    good = ((m.ids == -1) | (m.ids >= 4) | ((m.ids == 3) & ~broken))
    assert bool(good.any())
    assert torch.equal(m.y[:T][good], clean[:T][good])
    assert bool(m.y[:T][m.ids == 0].isnan().all()) and bool(m.y[:T][m.ids == 2].isnan().all())
    assert not bool(torch.isfinite(m.y[:T][broken]).any())
    # the adapter with non-finite weights: exactly its outputs that meet one are not finite, the others are right
    own = m.ids == 1
    if bool(own.any()):
        bad_out = (~torch.isfinite(m.b[1].float())).any(1)
        got = m.y[:T][own]
        assert not bool(torch.isfinite(got[:, bad_out]).any())
        want, bound = du.lora(m.x[own], m.w, m.a, torch.nan_to_num(m.b, nan=0.0, posinf=0.0, neginf=0.0), m.scale, m.ids[own])
        du.assert_within(got[:, ~bad_out], want[:, ~bad_out], bound[:, ~bad_out], "finite outputs")
        nan_out = m.b[1].isnan().any(1)
        assert bool(got[:, nan_out].isnan().all())


@pytest.mark.parametrize("T,mix", [(1, "one"), (48, "mixed"), (400, "runs"), (1500, "mixed")])
def test_the_same_call_gives_the_same_bits(T, mix):
    m = Linear(T, 512, 2048, 8, 32, mix)
    outs = []
    for _ in range(3):
        m.ws.fill_(255)                  # stale workspaces are never read (0xffff is a NaN)
        m.run()
        m.done()
        outs.append(m.y.clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_a_token_does_not_depend_on_its_neighbours_order():
    """The adapters' part of a token is the same whichever requests lie around it (the engines add it in the same
    accumulator, so only sums of the same length are compared: one engine, one tile)."""
    m = Linear(40, 256, 384, 5, 16, "mixed", seed=21)
    m.run()
    m.done()
    first = m.y.clone()
    p = torch.randperm(40, generator=torch.Generator().manual_seed(1)).cuda()
    m.x, m.ids = m.x[p].contiguous(), m.ids[p].contiguous()
    m.run()
    m.done()
    want, bound = du.lora(m.x, m.w, m.a, m.b, m.scale, m.ids)
    assert bool(((m.y[:40].double() - first[:40][p].double()).abs() <= 2 * bound).all())


def test_two_streams_at_once():
    ms = [Linear(T, 512, 2048, 6, 32, mix, seed=T) for T, mix in ((30, "mixed"), (1200, "runs"))]
    for m in ms:
        m.run()
        m.done()
        m.want, m.stream = m.y.clone(), torch.cuda.Stream()
        m.y.fill_(CANARY)
    torch.cuda.synchronize()
    for _ in range(10):
        for m in ms:
            m.run(m.stream)
    torch.cuda.synchronize()
    assert all(torch.equal(m.y, m.want) for m in ms) and ftm.ftm_device_status(True) == 0


@pytest.mark.parametrize("T", [20, 900])
def test_captured_and_replayed_with_other_requests(T):
    m = Linear(T, 256, 2048, 7, 16, "runs")
    m.run()
    m.done()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        m.run()
    for mix in ("mixed", "none", "distinct", "runs"):
        m.ids.copy_(adapters_of(T, 7, mix, seed=2))
        m.x.copy_(normal(77, T, 256))
        graph.replay()
        m.done()
        m.check()


def test_offsets_beyond_32_bits():
    """Pools and rows that end beyond 2^32 bytes from their start: the last adapter, the last rows."""
    T, d_in, d_out, n, rank = 6, 8192, 128, 4400, 64
    m = Linear(T, d_in, d_out, 1, rank, "one", seed=8)
    a = torch.zeros(n, rank, d_in, dtype=torch.bfloat16, device="cuda")          # 4.6 GB
    assert a.numel() > 2 ** 31
    b = torch.zeros(n, d_out, rank, dtype=torch.bfloat16, device="cuda")
    a[n - 1], b[n - 1] = m.a[0], m.b[0]
    scale = torch.full((n,), 1.5, device="cuda")
    m.a, m.b, m.scale = a, b, scale
    m.D.n_adapters = n
    m.ids = torch.tensor([n - 1, -1, n - 1, 0, n - 1, n - 2], dtype=torch.int32, device="cuda")
    m.run()
    m.done()
    m.check()
    del a, b, m
    for T, ld in ((5, 1 << 29), (300, 1 << 23)):                                  # few tokens and CTA pairs
        m = Linear(T, 256, 8200 if T > 5 else 128, 3, 16, "mixed", seed=4)
        big = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)
        y = big[:, :m.D.d_out]
        ftm.ftm_lora_linear(m.D, m.x, T, m.w, m.a, m.b, m.scale, m.ids, y, m.ws, m.ws.numel(), ldy=ld)
        m.done()
        want, bound = du.lora(m.x, m.w, m.a, m.b, m.scale, m.ids)
        du.assert_within(y, want, bound, "far rows")
        del big, y


def test_no_tokens_and_wrong_memory():
    m = Linear(4, 256, 128, 2, 16)
    ftm.ftm_lora_linear(m.D, None, 0, None, None, None, None, None, None, None, 0)
    for name in ("x", "w", "a", "b", "scale", "ids", "y"):
        bad = Linear(4, 256, 128, 2, 16)
        setattr(bad, name, getattr(bad, name).cpu())
        with pytest.raises(ftm.FtmError) as e:
            bad.run()
        assert e.value.status == 1 and "not memory of the current device" in str(e.value)
    m.run()
    m.done()
    m.check()


@pytest.mark.parametrize("T", [7, 150, 1300])
def test_served_block_with_adapters_and_its_training_step(T):
    """As they are used: a shared projection with every request's adapter feeds the dense gated block, in one stream
    without a wait between them; each stage is checked on what the stage before really gave."""
    d_in, d, I = 384, 512, 256
    m = Linear(T, d_in, d, 5, 16, "runs", seed=31, std=0.1)
    L = ftm.LayerDesc(d, 1, 1, I, 0, 1, ftm.FTM_BF16, 0)
    bank, dy = normal(41, 3 * I * d, std=0.05), normal(42, T, d)
    y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    pre = torch.empty(T, 2 * I, dtype=torch.bfloat16, device="cuda")
    dx, dbank = torch.empty_like(y), torch.empty_like(bank)
    ws = torch.empty(max(ftm.ftm_gated_ffn_workspace_bytes(L, T), ftm.ftm_gated_ffn_backward_workspace_bytes(L, T)),
                     dtype=torch.uint8, device="cuda")
    for _ in range(3):
        m.run()
        ftm.ftm_gated_ffn(L, ftm.FTM_ACT_SILU, m.y, T, bank, pre, y, ws, ws.numel())
        ftm.ftm_gated_ffn_backward(L, ftm.FTM_ACT_SILU, m.y, T, bank, pre, dy, dx, dbank, ws, ws.numel())
    m.done()
    m.check()
    mid = m.y[:T]
    (g, u, want), (eg, eu, ey) = du.block_forward(mid, bank, d, I, "silu")
    du.assert_within(y, want, ey, "block")
    du.assert_within(pre[:, :I], g, eg, "g")
    (wx, ww, wd), (ex, ew, ed) = du.block_backward(mid, bank, pre, dy, d, I, "silu")
    du.assert_within(dx, wx, ex, "dx")
    du.assert_within(dbank[:2 * I * d].view(2 * I, d), ww, ew, "dw_gu")
    du.assert_within(dbank[2 * I * d:].view(d, I), wd, ed, "dw_d")


@pytest.mark.parametrize("T,d_in,d_out", [(4, 264, 256), (7, 264, 256), (24, 264, 256), (100, 256, 4096), (640, 520, 2048), (2500, 264, 2048)])
def test_an_infinite_low_rank_value_meets_infinite_weights(T, d_in, d_out):
    """s (x A^T) beyond the largest bf16 is an infinity of its sign; with weights of B that are infinite, and others
    that are not, of one sign an output is that infinity, of both NaN, on every engine."""
    m = Linear(T, d_in, d_out, 4, 24, "mixed", seed=5)
    m.ids[0], m.ids[T - 1] = 2, -1
    m.x.abs_()
    m.a[2].abs_()                        # x A^T is above 1 everywhere, times 3e38 beyond the range
    m.b[2].abs_()
    m.scale[2] = 3e38
    inf = float("inf")
    m.b[2, 0::7, 5] = inf                # outputs 0 mod 7: +inf + (inf * inf); 1 mod 7: -inf everywhere; 2 mod 7: both; others inf * finite
    m.b[2, 1::7] *= -1
    m.b[2, 1::7, 23] = -inf
    m.b[2, 2::7, 3] = -inf
    m.b[2, 3::7, 9] = float("nan")
    m.run()
    m.done()
    own = m.ids == 2
    assert bool((m.x[own].double() @ m.a[2].double().T > 2.0).all())
    got = m.y[:T].double()
    want = torch.full((d_out,), inf, dtype=torch.float64, device="cuda")
    want[1::7], want[2::7], want[3::7] = -inf, float("nan"), float("nan")
    assert torch.equal(got[own].nan_to_num(nan=1.0), want.nan_to_num(nan=1.0).expand(int(own.sum()), d_out))
    assert torch.equal(got[own].isnan(), want.isnan().expand(int(own.sum()), d_out))
    ids = torch.where(own, torch.full_like(m.ids, -1), m.ids)
    ref, bound = du.lora(m.x, m.w, m.a, m.b, m.scale, ids)
    du.assert_within(got[~own], ref[~own], bound[~own], "other requests")


@pytest.mark.parametrize("T,d_in,d_out,rank,scaled", [(1, 2048, 256, 128, True), (4, 512, 520, 32, False), (8, 264, 136, 16, True)])
def test_one_launch_rounds_once(T, d_in, d_out, rank, scaled):
    """Up to 8 tokens in one launch: sums in fp32 from end to end and one rounding, of y.  The adapter's part cancels
    almost wholly over the rank, so that a rounding of s (x A^T) would be seen."""
    m = Linear(T, d_in, d_out, T, rank, "distinct", seed=7, scaled=scaled, std=1.0)
    m.w.zero_()
    m.a[:, 1::2] = m.a[:, ::2] * 1.0625          # neighbouring values of v: v and 1.0625 v
    m.a[:, 1::2] = m.a[:, 1::2].to(torch.bfloat16)
    m.b[:, :, 1::2] = -m.b[:, :, ::2]
    m.run()
    m.done()
    X = m.x.double()
    A, B = m.a.double()[m.ids.long()], m.b.double()[m.ids.long()]
    s = torch.ones(T, 1, device="cuda", dtype=torch.float64) if m.scale is None else m.scale.double()[m.ids.long()].unsqueeze(1)
    v = s * torch.einsum("tk,trk->tr", X, A)
    want = torch.einsum("tr,tor->to", v, B)
    # v: sums of K products and a multiplication; y: a sum of rank products and a rounding
    ev = (du.gamma(d_in) + 2.0 ** -23) * s.abs() * torch.einsum("tk,trk->tr", X.abs(), A.abs())
    ey = torch.einsum("tr,tor->to", ev + du.gamma(rank) * (v.abs() + ev), B.abs())
    du.assert_within(m.y[:T], want, ey + du.U * (want.abs() + ey), "y")
    assert float((want - m.y[:T].double()).norm() / want.norm()) <= du.U      # one rounding's worst case


@pytest.mark.parametrize("T,d_in,d_out,rank", [
    (6, 264, 200, 16), (24, 320, 256, 40), (60, 1000, 512, 24), (100, 320, 4096, 40), (500, 4096, 2560, 16),
    (640, 520, 2048, 40), (900, 512, 2048, 16), (2500, 320, 2048, 40)])
def test_what_other_requests_hold_changes_no_bit(T, d_in, d_out, rank):
    """With the ids as they are, every other value (rows of other adapters' tokens, the adapters, their scales) may
    change: a token's bits stay.  One launch, few tokens split along K, CTA pairs split along K (640, 900, 500) and not."""
    m = Linear(T, d_in, d_out, 6, rank, "mixed", seed=13)
    m.ids[1] = 3
    m.run()
    m.done()
    m.check()
    first = m.y.clone()
    own = m.ids == 3
    other = torch.arange(6, device="cuda") != 3
    for seed in (100, 200):
        m.x[~own] = normal(seed, T, d_in, std=3.0)[~own]
        m.a[other] = normal(seed + 1, *m.a.shape, std=0.2)[other]
        m.b[other] = normal(seed + 2, *m.b.shape, std=2.0)[other]
        m.scale[other] *= -1.7
        m.run()
        m.done()
        m.check()
        assert torch.equal(m.y[:T][own], first[:T][own]) and not torch.equal(m.y, first)


# CTA pairs, one tile to a cluster whose pairs split the depth: more than 74 tiles of 128 x 128 (else the few-token
# engine), at most 37 of 256 x 256, d_in >= 512; 20 and 24 tiles in clusters of 3 or 2 pairs, 32 of 2
SPLIT_PAIRS = [(500, 4096, 2560), (640, 520, 2048), (900, 512, 2048)]


@pytest.mark.parametrize("T,d_in,d_out", SPLIT_PAIRS)
@pytest.mark.parametrize("n,rank,mix", [(6, 40, "mixed"), (3, 128, "runs"), (1, 16, "one"), (4, 64, "none"), (64, 8, "distinct")])
def test_projection_split_over_pairs(T, d_in, d_out, n, rank, mix):
    m = Linear(T, d_in, d_out, n, rank, mix, seed=T + rank)
    outs = []
    for _ in range(3):
        m.ws.fill_(255)
        m.run()
        m.done()
        m.check()
        outs.append(m.y.clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("T,d_in,d_out", SPLIT_PAIRS)
@pytest.mark.parametrize("broken", range(6))
def test_requests_are_isolated_where_pairs_split_the_depth(T, d_in, d_out, broken):
    """One adapter after the other (each lies elsewhere in the tiles' lists, so another pair feeds its slices) has
    infinities and NaN in B: in every fifth output, so in columns that each of the cluster's pairs finishes."""
    m = Linear(T, d_in, d_out, 6, 40, "mixed", seed=11)
    m.run()
    m.done()
    clean = m.y.clone()
    r = (7 * broken) % 40                # a different slice of 16 for different adapters
    m.b[broken, ::5, r] = float("inf")
    m.b[broken, 1::5, 39 - r] = float("nan")
    m.b[broken, 2::5, (r + 16) % 40] = -float("inf")
    m.run()
    m.done()
    own = m.ids == broken
    assert torch.equal(m.y[:T][~own], clean[:T][~own]) and torch.equal(m.y[T:], clean[T:])
    got = m.y[:T][own].double()
    v = (m.x[own].double() @ m.a[broken].double().T) * m.scale[broken].double()
    ev = (du.gamma(d_in) + 2.0 ** -23) * (m.x[own].double().abs() @ m.a[broken].double().abs().T) * m.scale[broken].double().abs()
    for at, k, sign in ((0, r, 1.0), (2, (r + 16) % 40, -1.0)):
        sure = v[:, k].abs() > ev[:, k]                    # the others are zero within the error of their sums
        assert int(sure.sum()) > 0.9 * sure.numel() and not bool(torch.isfinite(got[:, at::5]).any())
        far = torch.full_like(got[sure, at::5], sign * float("inf"))
        assert torch.equal(got[sure, at::5], far * v[sure, k:k + 1].sign())
    assert bool(got[:, 1::5].isnan().all())
    finite = torch.arange(d_out, device="cuda") % 5 > 2
    assert torch.equal(m.y[:T][own][:, finite], clean[:T][own][:, finite])


@pytest.mark.parametrize("T,d_in,d_out", SPLIT_PAIRS)
def test_split_over_pairs_captured_strided_and_on_two_streams(T, d_in, d_out):
    m = Linear(T, d_in, d_out, 5, 24, "runs", seed=17)
    big = torch.full((T + 2, d_in + d_out + 48), CANARY, dtype=torch.bfloat16, device="cuda")
    x, y = big[:T, 16:16 + d_in], big[:T, d_in + 32:d_in + 32 + d_out]

    def run(stream=None):
        ftm.ftm_lora_linear(m.D, x, T, m.w, m.a, m.b, m.scale, m.ids, y, m.ws, m.ws.numel(), stream, ldx=big.stride(0),
                            ldy=big.stride(0))
    x.copy_(m.x)
    run()
    m.done()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        run()
        run()
    for mix in ("mixed", "none", "distinct", "runs"):
        m.ids.copy_(adapters_of(T, 5, mix, seed=2))
        m.x = normal(78, T, d_in)
        x.copy_(m.x)
        before = big.clone()
        y.fill_(CANARY)
        graph.replay()
        m.done()
        want, bound = du.lora(m.x, m.w, m.a, m.b, m.scale, m.ids)
        du.assert_within(y, want, bound, "y")
        before[:T, d_in + 32:d_in + 32 + d_out] = y
        assert torch.equal(big, before)
    other = Linear(T + 130, d_in, d_out, 4, 16, "mixed", seed=18)
    keep, streams = y.clone(), (torch.cuda.Stream(), torch.cuda.Stream())
    torch.cuda.synchronize()
    for _ in range(10):
        run(streams[0])
        other.run(streams[1])
    other.done()
    other.check()
    assert torch.equal(y, keep)


@pytest.mark.parametrize("T,d_in,d_out,n,rank,mix", [(9, 4096, 9728, 4, 16, "distinct"), (32, 512, 9600, 32, 16, "distinct"),
                                                     (64, 4096, 9728, 6, 40, "mixed"), (128, 264, 10248, 3, 128, "runs"),
                                                     (5, 520, 20480, 5, 16, "mixed")])
def test_few_tokens_on_wide_projections(T, d_in, d_out, n, rank, mix):
    m = Linear(T, d_in, d_out, n, rank, mix, seed=T)
    m.run()
    m.done()
    m.check()
