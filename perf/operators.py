"""The operators beside the routed experts, as they are measured: the dense gated feed-forward block of an
MoE model (its leading dense layers, its shared expert) forward and as a training step, and a projection
that many requests share while each of them brings its own low-rank adapter.

Formulas (x [T][d], weights row-major, one row per output):

  gated block   g = x Wg^T, u = x Wu^T, h = act(g) * u, y = h Wd^T
                act = silu: z sigmoid(z); gelu: z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))
  its backward  dh = dy Wd, dWd = dy^T h, dg = dh * u * act'(g), du = dh * act(g),
                dWg = dg^T x, dWu = du^T x, dx = dg Wg + du Wu
  adapters      y[t] = x[t] W^T + s[a] (x[t] A[a]^T) B[a]^T with a = adapter[t]; a = -1: the shared part alone
"""
import math

import torch

own = False

GELU_C = math.sqrt(2.0 / math.pi)


def listed():
    return [
        # one token through a 35B-class shared expert: pure latency, 9.4 MB of weights
        {"name": "ffn_token", "op": "ffn", "act": "silu", "T": 1, "d": 2048, "I": 768},
        # a decode batch through a 753B-class dense block: bound by the 75 MB of weights
        {"name": "ffn_decode", "op": "ffn", "act": "silu", "T": 32, "d": 6144, "I": 2048},
        # a packed prompt of odd length, GELU form
        {"name": "ffn_prompt", "op": "ffn", "act": "gelu", "T": 5003, "d": 4096, "I": 2048},
        # fine-tuning on one short odd batch of a small block
        {"name": "train_short", "op": "train", "act": "gelu", "T": 333, "d": 2048, "I": 768},
        # an ordinary training micro-batch
        {"name": "train_batch", "op": "train", "act": "silu", "T": 4096, "d": 4096, "I": 2048},
        # the largest: a long-context micro-batch of the widest block
        {"name": "train_long", "op": "train", "act": "silu", "T": 16384, "d": 6144, "I": 2048},
        # one token of one request
        {"name": "lora_token", "op": "lora", "T": 1, "d_in": 2048, "d_out": 2048, "rank": 8, "adapters": 4,
         "requests": 1},
        # a decode batch in which every token is another request's
        {"name": "lora_decode", "op": "lora", "T": 64, "d_in": 4096, "d_out": 4096, "rank": 16, "adapters": 32,
         "requests": 64},
        # a wide decode batch over a narrowing projection, large rank
        {"name": "lora_wide", "op": "lora", "T": 256, "d_in": 6144, "d_out": 2048, "rank": 64, "adapters": 16,
         "requests": 256},
        # odd sizes everywhere
        {"name": "lora_odd", "op": "lora", "T": 77, "d_in": 1000, "d_out": 1736, "rank": 24, "adapters": 5,
         "requests": 9},
        # packed prompts of a few requests
        {"name": "lora_prompts", "op": "lora", "T": 2500, "d_in": 2048, "d_out": 4096, "rank": 32, "adapters": 8,
         "requests": 7},
        # a full prefill batch
        {"name": "lora_prefill", "op": "lora", "T": 8192, "d_in": 4096, "d_out": 6144, "rank": 16, "adapters": 16,
         "requests": 12},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "train", "lora"])
    if op == "lora":
        T = _log_int(rng, 1, 8192)
        d_in, d_out = 8 * _log_int(rng, 32, 768), 8 * _log_int(rng, 32, 768)
        requests = T if rng.random() < 0.4 and T <= 512 else min(T, _log_int(rng, 1, 64))
        return {"op": op, "T": T, "d_in": d_in, "d_out": d_out, "rank": 8 * rng.randint(1, 16),
                "adapters": _log_int(rng, 1, 32), "requests": requests}
    return {"op": op, "act": rng.choice(["silu", "gelu"]), "T": _log_int(rng, 1 if op == "ffn" else 16, 16384),
            "d": 128 * _log_int(rng, 2, 48), "I": 128 * _log_int(rng, 1, 16)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)

    T = case["T"]
    s = {"op": case["op"], "T": T}
    if case["op"] == "lora":
        n, r, d_in, d_out, q = (case[k] for k in ("adapters", "rank", "d_in", "d_out", "requests"))
        s["sizes"] = (d_in, d_out, n, r)
        s["x"] = normal(T, d_in)
        s["w"] = normal(d_out, d_in, std=0.02)
        s["a"] = normal(n, r, d_in, std=0.02)
        s["b"] = normal(n, d_out, r, std=0.02)
        s["scale"] = 0.5 + 1.5 * torch.rand(n, generator=gen, device="cuda")
        # requests lie one behind the other, of uneven lengths; about one in eight has no adapter
        cuts = torch.randperm(T - 1, generator=gen, device="cuda")[:q - 1].sort().values + 1 if q > 1 else None
        of_request = torch.randint(0, n, (q,), generator=gen, device="cuda")
        none = torch.rand(q, generator=gen, device="cuda") < 0.125
        of_request = torch.where(none & (q > 1), torch.full_like(of_request, -1), of_request)
        at = torch.arange(T, device="cuda")
        request = torch.searchsorted(cuts, at, right=True) if cuts is not None else torch.zeros_like(at)
        s["adapter"] = of_request[request].to(torch.int32)
        s["y"] = torch.empty(T, d_out, dtype=torch.bfloat16, device="cuda")
        return s
    d, I = case["d"], case["I"]
    s["act"], s["sizes"] = case["act"], (d, I)
    s["x"] = normal(T, d)
    # one bank: the 2I gate and up rows, then the down projection
    s["bank"] = normal(3 * I * d, std=0.02)
    s["y"] = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    if case["op"] == "train":
        s["dy"] = normal(T, d)
        s["pre"] = torch.empty(T, 2 * I, dtype=torch.bfloat16, device="cuda")
        s["dx"] = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
        s["dbank"] = torch.empty(3 * I * d, dtype=torch.bfloat16, device="cuda")
    return s


def _workspace(s, nbytes):
    # as a user's program does: one buffer per plan, made when it is first needed
    if "ws" not in s:
        s["ws"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return s["ws"]


def _run_own(s):
    import expert_offloaded_edge_b200 as ftm

    T = s["T"]
    if s["op"] == "lora":
        d_in, d_out, n, r = s["sizes"]
        D = ftm.LoraDesc(d_in, d_out, n, r, ftm.FTM_BF16, 0)
        ws = _workspace(s, ftm.ftm_lora_workspace_bytes(D, T))
        ftm.ftm_lora_linear(D, s["x"], T, s["w"], s["a"], s["b"], s["scale"], s["adapter"], s["y"], ws, ws.numel())
        return s["y"]
    d, I = s["sizes"]
    L = ftm.LayerDesc(d, 1, 1, I, 0, 1, ftm.FTM_BF16, 0)
    act = ftm.FTM_ACT_SILU if s["act"] == "silu" else ftm.FTM_ACT_GELU_TANH
    if s["op"] == "ffn":
        ws = _workspace(s, ftm.ftm_gated_ffn_workspace_bytes(L, T))
        ftm.ftm_gated_ffn(L, act, s["x"], T, s["bank"], None, s["y"], ws, ws.numel())
        return s["y"]
    ws = _workspace(s, max(ftm.ftm_gated_ffn_workspace_bytes(L, T), ftm.ftm_gated_ffn_backward_workspace_bytes(L, T)))
    ftm.ftm_gated_ffn(L, act, s["x"], T, s["bank"], s["pre"], s["y"], ws, ws.numel())
    ftm.ftm_gated_ffn_backward(L, act, s["x"], T, s["bank"], s["pre"], s["dy"], s["dx"], s["dbank"], ws, ws.numel())
    return {"y": s["y"], "dx": s["dx"], "dw_gu": s["dbank"][:2 * I * d].view(2 * I, d),
            "dw_d": s["dbank"][2 * I * d:].view(d, I)}


def run(s):
    if own:
        return _run_own(s)
    x = s["x"].float()
    if s["op"] == "lora":
        d_in, d_out, n, r = s["sizes"]
        # every adapter's rows at once, those of other adapters than the token's zeroed
        mine = s["adapter"].unsqueeze(1) == torch.arange(n, device=x.device)
        v = (x @ s["a"].float().view(n * r, d_in).t()).view(-1, n, r)
        v = torch.where(mine.unsqueeze(2), v * s["scale"].view(1, n, 1), torch.zeros_like(v))
        y = x @ s["w"].float().t()
        y = y + v.reshape(-1, n * r) @ s["b"].float().transpose(1, 2).reshape(n * r, d_out)
        return y.to(torch.bfloat16)
    d, I = s["sizes"]
    w_gu = s["bank"][:2 * I * d].view(2 * I, d).float()
    w_d = s["bank"][2 * I * d:].view(d, I).float()
    gu = x @ w_gu.t()
    g, u = gu[:, :I], gu[:, I:]
    if s["act"] == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        a, da = g * sig, sig * (1.0 + g * (1.0 - sig))
    else:
        th = torch.tanh(GELU_C * (g + 0.044715 * g * g * g))
        a = 0.5 * g * (1.0 + th)
        da = 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * GELU_C * (1.0 + 3 * 0.044715 * g * g)
    h = a * u
    y = h @ w_d.t()
    if s["op"] == "ffn":
        return y.to(torch.bfloat16)
    dy = s["dy"].float()
    dh = dy @ w_d
    dgu = torch.cat([dh * u * da, dh * a], dim=1)
    return {"y": y.to(torch.bfloat16), "dx": (dgu @ w_gu).to(torch.bfloat16), "dw_gu": (dgu.t() @ x).to(torch.bfloat16),
            "dw_d": (dy.t() @ h).to(torch.bfloat16)}


def work(case):
    T = case["T"]
    if case["op"] == "lora":
        d_in, d_out, n, r = (case[k] for k in ("d_in", "d_out", "adapters", "rank"))
        used = min(n, case["requests"])
        return {"bytes": 2 * (T * d_in + d_out * d_in + used * r * (d_in + d_out) + T * d_out) + 4 * T + 4 * n,
                "flops": 2 * T * d_in * d_out + 2 * T * r * (d_in + d_out)}
    d, I = case["d"], case["I"]
    if case["op"] == "ffn":
        return {"bytes": 2 * (2 * T * d + 3 * I * d), "flops": 6 * T * d * I}
    # x, dy and the weights in; y, dx and the weights' gradients out
    return {"bytes": 2 * (4 * T * d + 6 * I * d), "flops": 18 * T * d * I}


def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "lora":
        ids = s["adapter"].long()
        y = torch.mm(s["x"].to(f), s["w"].to(f).T)
        for a in range(case["adapters"]):
            rows = torch.nonzero(ids == a).flatten()
            if rows.numel():
                low = s["x"][rows].to(f).mm(s["a"][a].to(f).T)
                y[rows] += float(s["scale"][a]) * low.mm(s["b"][a].to(f).T)
        return y
    d, I, T = case["d"], case["I"], case["T"]
    w_g, w_u, w_d = (s["bank"][k * I * d:(k + 1) * I * d].to(f) for k in range(3))
    w_g, w_u, w_d = w_g.view(I, d), w_u.view(I, d), w_d.view(d, I)
    x = s["x"].to(f)
    g = torch.mm(x, w_g.T)
    u = torch.mm(x, w_u.T)
    if case["act"] == "silu":
        p = torch.sigmoid(g)
        act = g * p
        slope = p + act * (1 - p)
    else:
        inner = GELU_C * g * (1 + 0.044715 * g.square())
        c = torch.tanh(inner)
        act = g * (1 + c) / 2
        slope = (1 + c) / 2 + g / 2 / torch.cosh(inner).square() * GELU_C * (1 + 0.134145 * g.square())
    h = act * u
    y = torch.mm(h, w_d.T)
    if case["op"] == "ffn":
        return y
    dy = s["dy"].to(f)
    dh = torch.mm(dy, w_d)
    dg, du = dh * u * slope, dh * act
    return {"y": y, "dx": torch.mm(dg, w_g) + torch.mm(du, w_u),
            "dw_gu": torch.cat([torch.mm(dg.T, x), torch.mm(du.T, x)]), "dw_d": torch.mm(dy.T, h)}
