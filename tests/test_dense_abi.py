"""CPU checks of the dense operators' C ABI: what they refuse before touching a GPU, and that the 64-bit
references of their GPU tests are right (the gradients against central differences)."""
import ctypes

import pytest
import torch

import expert_offloaded_edge_b200 as ftm
from tests import dense_util as du

BF16 = ftm.FTM_BF16
A = 0x7000_0000_0000          # addresses that are never dereferenced
STEP = 0x1_0000_0000


def layer(**kw):
    f = dict(d=256, E=4, k=2, I=128, has_shared=1, S=4, wdtype=BF16, reserved=0)
    f.update(kw)
    return ftm.LayerDesc(**f)


def lora(**kw):
    f = dict(d_in=256, d_out=128, n_adapters=4, rank=16, wdtype=BF16, reserved=0)
    f.update(kw)
    return ftm.LoraDesc(**f)


def forward(L, act=0, x=A, T=4, bank=A + STEP, pre=None, y=A + 2 * STEP, ws=A + 3 * STEP, n=1 << 20):
    return ftm.library().ftm_gated_ffn(ctypes.byref(L), act, x, T, bank, pre, y, ws, n, None)


def backward(L, act=0, x=A, T=4, bank=A + STEP, pre=A + 2 * STEP, dy=A + 3 * STEP, dx=A + 4 * STEP,
             dbank=A + 5 * STEP, ws=A + 6 * STEP, n=1 << 20):
    return ftm.library().ftm_gated_ffn_backward(ctypes.byref(L), act, x, T, bank, pre, dy, dx, dbank, ws, n, None)


def linear(D, x=A, ldx=None, T=4, w=A + STEP, a=A + 2 * STEP, b=A + 3 * STEP, scale=None, ids=A + 4 * STEP,
           y=A + 5 * STEP, ldy=None, ws=A + 6 * STEP, n=1 << 20):
    return ftm.library().ftm_lora_linear(ctypes.byref(D), x, D.d_in if ldx is None else ldx, T, w, a, b, scale, ids, y,
                                         D.d_out if ldy is None else ldy, ws, n, None)


def refused(status, code, text):
    assert status == code, (status, ftm.ftm_last_error())
    assert text in ftm.ftm_last_error(), ftm.ftm_last_error()


@pytest.mark.parametrize("call", [forward, backward])
def test_block_refusals(call):
    refused(call(layer(d=100)), 1, "multiple of 128")
    refused(call(layer(reserved=1)), 1, "reserved")
    for wd in (ftm.FTM_F32, ftm.FTM_FP8_E4M3_B128, ftm.FTM_NVFP4, ftm.FTM_MXFP4):
        refused(call(layer(d=256, I=256, wdtype=wd)), 2, "bf16 banks only")
    refused(call(layer(d=1 << 21)), 2, "above")
    refused(call(layer(), act=2), 1, "activation")
    refused(call(layer(), act=-1), 1, "activation")
    refused(call(layer(), T=-1), 1, "negative")
    refused(call(layer(), T=1 << 30), 1, "too large")
    refused(call(layer(), n=16), 1, "needed")
    refused(call(layer(), ws=None), 1, "workspace is NULL")
    refused(call(layer(), ws=A + 3 * STEP + 64), 1, "256-byte")
    for arg in ("x", "bank"):
        refused(call(layer(), **{arg: None}), 1, f"{arg} is NULL")
        refused(call(layer(), **{arg: A + STEP + 8}), 1, f"{arg} is not 16-byte aligned")


def test_forward_refusals():
    refused(forward(layer(), y=None), 1, "y is NULL")
    refused(forward(layer(), y=A), 1, "y overlaps x")
    refused(forward(layer(), y=A + 4 * 256 * 2 - 16), 1, "y overlaps x")
    refused(forward(layer(), pre=A + STEP), 1, "overlaps")
    refused(forward(layer(), ws=A), 1, "overlaps")
    assert forward(layer(), T=0, x=None, bank=None, y=None, ws=None, n=0) == 0      # no-op


def test_backward_refusals():
    refused(backward(layer(), pre=None), 1, "pre is NULL")
    refused(backward(layer(), dy=None), 1, "dy is NULL")
    refused(backward(layer(), dx=None, dbank=None), 1, "both NULL")
    refused(backward(layer(), dx=A), 1, "dx overlaps x")
    refused(backward(layer(), dx=A + 3 * STEP), 1, "dx overlaps dy")
    refused(backward(layer(), dbank=A + STEP), 1, "dbank overlaps bank")
    refused(backward(layer(), dbank=A + 2 * STEP), 1, "dbank overlaps pre")
    assert backward(layer(), T=0, dbank=None) == 0                                  # nothing to set
    assert ftm.ftm_gated_ffn_backward_workspace_bytes(layer(), 4) > ftm.ftm_gated_ffn_workspace_bytes(layer(), 4) > 0
    assert ftm.ftm_gated_ffn_workspace_bytes(layer(wdtype=ftm.FTM_F32), 4) == 0


@pytest.mark.parametrize("field,value,code,text", [
    ("d_in", 0, 1, "d_in"), ("d_in", 12, 1, "d_in"), ("d_in", 1 << 21, 1, "d_in"), ("d_out", 4, 1, "d_out"),
    ("d_out", -8, 1, "d_out"), ("rank", 0, 1, "rank"), ("rank", 12, 1, "rank"), ("rank", 136, 1, "rank"),
    ("n_adapters", 0, 1, "n_adapters"), ("n_adapters", 65537, 1, "n_adapters"), ("reserved", 1, 1, "reserved"),
    ("wdtype", 9, 1, "wdtype"), ("wdtype", ftm.FTM_F32, 2, "bf16 only")])
def test_lora_desc_refusals(field, value, code, text):
    refused(linear(lora(**{field: value})), code, text)
    assert ftm.ftm_lora_workspace_bytes(lora(**{field: value}), 4) == 0


def test_lora_refusals():
    D = lora()
    refused(linear(D, ldx=248), 1, "ldx")
    refused(linear(D, ldx=260), 1, "ldx")
    refused(linear(D, ldy=120), 1, "ldy")
    refused(linear(D, ldy=132), 1, "ldy")
    refused(linear(D, T=-1), 1, "negative")
    refused(linear(D, n=16), 1, "needed")
    refused(linear(D, ws=A + 6 * STEP + 16), 1, "256-byte")
    for arg in ("x", "w", "y"):
        refused(linear(D, **{arg: None}), 1, f"{arg} is NULL")
        refused(linear(D, **{arg: A + 7 * STEP + 2}), 1, f"{arg} is not 16-byte aligned")
    refused(linear(D, a=None), 1, "lora_a is NULL")
    refused(linear(D, b=None), 1, "lora_b is NULL")
    refused(linear(D, ids=None), 1, "adapter_ids is NULL")
    refused(linear(D, ids=A + 4 * STEP + 2), 1, "adapter_ids is not 4-byte aligned")
    refused(linear(D, scale=A + 7 * STEP + 1), 1, "scale is not 4-byte aligned")
    refused(linear(D, y=A), 1, "y overlaps x")
    refused(linear(D, y=A + STEP + 128), 1, "y overlaps w")
    refused(linear(D, y=A + 4 * STEP), 1, "y overlaps adapter_ids")
    refused(linear(D, ids=A + 5 * STEP - 4), 1, "y overlaps adapter_ids")       # its last three entries
    # column slices of one matrix: 256 + 128 columns of 384 share no byte, 16 columns earlier they do
    refused(linear(D, ldx=384, ldy=384, y=A + 2 * 240), 1, "y overlaps x")
    assert "overlap" not in (linear(D, ldx=384, ldy=384, y=A + 2 * 256) and ftm.ftm_last_error())
    assert "overlap" not in (linear(D, ldx=384, ldy=384, x=A + 2 * 128, y=A) and ftm.ftm_last_error())
    assert linear(D, T=0, x=None, w=None, y=None, ws=None, n=0) == 0                # no-op


def test_host_memory_is_refused():
    """Buffers that lie in host memory (or, here, that no device knows) never reach a kernel."""
    assert forward(layer()) != 0 and backward(layer()) != 0 and linear(lora()) != 0


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_reference_gradients_against_differences(act):
    g = torch.Generator().manual_seed(3)
    T, d, I = 5, 6, 7

    def rand(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    x, bank, dy = rand(T, d), 0.7 * rand(3 * I * d), rand(T, d)

    def loss(x, bank):
        wg, wu, wd = (bank[k * I * d:(k + 1) * I * d] for k in range(3))
        z = x @ wg.view(I, d).T
        a, _ = du.activation(z, act)
        return float(((a * (x @ wu.view(I, d).T)) @ wd.view(d, I).T * dy).sum())

    wg, wu, _ = du.split_bank(bank, d, I)
    pre = torch.cat([x @ wg.T, x @ wu.T], 1)
    (dx, dw, dwd), _ = du.block_backward(x, bank, pre, dy, d, I, act)
    dbank = torch.cat([dw.flatten(), dwd.flatten()])
    for _ in range(8):
        vx, vb = rand(T, d), rand(3 * I * d)
        e = 1e-5
        num = (loss(x + e * vx, bank + e * vb) - loss(x - e * vx, bank - e * vb)) / (2 * e)
        ana = float((dx * vx).sum() + (dbank * vb).sum())
        # central differences: the third derivative's e^2 and the rounding 2^-53 |loss| / e
        assert abs(num - ana) <= 1e-6 * (1 + abs(ana)) + 1e-7
    # and the activations' slope by itself, at the clamp's border too
    for z0 in (-20.0, -12.0, -3.0, -0.5, 0.0, 0.7, 4.0, 12.0, 20.0):
        z = torch.tensor([z0 - 1e-5, z0, z0 + 1e-5], dtype=torch.float64)
        a, s = du.activation(z, act)
        assert abs(float(a[2] - a[0]) / 2e-5 - float(s[1])) < 1e-8


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_the_norm_of_a_gradients_error_sees_a_block_left_out(act):
    """At 20000 tokens: roundings to bf16 where the kernels make them stay within du.NORM, and 64 tokens that a sum
    leaves out (its last, or any) do not, in either weight gradient."""
    g = torch.Generator().manual_seed(5)
    T, d, I = 20000, 24, 16

    def rand(*s, std=1.0):
        return (torch.randn(*s, generator=g) * std).to(torch.bfloat16)

    x, bank, dy, pre = rand(T, d), rand(3 * I * d, std=0.2), rand(T, d), rand(T, 2 * I)

    def bf(t):
        return t.to(torch.bfloat16).double()

    (dx, dw, dwd), _ = du.block_backward(x, bank, pre, dy, d, I, act)
    wg, wu, wd = du.split_bank(bank, d, I)
    z, u = pre[:, :I].double(), pre[:, I:].double()
    a, slope = du.activation(z, act)
    dh = dy.double() @ wd
    dgu, h = bf(torch.cat([dh * u * slope, dh * a], 1)), bf(a * u)
    assert du.norm_error(bf(dgu @ torch.cat([wg, wu])), dx) <= du.NORM
    assert du.norm_error(bf(dgu.T @ x.double()), dw) <= du.NORM
    assert du.norm_error(bf(dy.double().T @ h), dwd) <= du.NORM
    for lost in (slice(T - 64, T), slice(6400, 6464)):
        keep = torch.ones(T, dtype=torch.bool)
        keep[lost] = False
        assert du.norm_error(dgu[keep].T @ x[keep].double(), dw) > 3 * du.NORM
        assert du.norm_error(dy[keep].double().T @ h[keep], dwd) > 3 * du.NORM
