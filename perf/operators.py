"""The workloads of the few-token layer and of the per-request adapters.

Two operators are run here, each over the range of sizes it is used at:

``decode``   the whole routed-expert layer for a few tokens
             (``strata_moe_decode``): router, top-K softmax, int8 rounding of
             the input, gate/up + SwiGLU + int8 rounding of H, down, the
             weighted sum; optionally a shared expert, a router bias and the
             requests' adapters beside the layer.
``adapt``    low-rank adapters of many requests beside a projection they share
             (``strata_moe_adapt``): out[t] = y[t] + scale_a B_a (A_a x[t]) with
             a = ids[t], and out[t] = y[t] where ids[t] < 0.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from
a seed, ``run`` is one call.  With ``own`` false the call is spelled out in
elementary torch operations; with ``own`` true it goes through the library.
``exact`` evaluates the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32
CODE_ZERO = {"q2_sym": 1.5, "q2_0": 1.0}
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases
def _decode(name, T, H, E, K, I, fmt="q2_sym", shared=False, skewed=False, rank=0, adapters=0, dtype="bf16"):
    return dict(name=name, op="decode", T=T, H=H, E=E, K=K, I=I, fmt=fmt, shared=shared, skewed=skewed, rank=rank,
                adapters=adapters, dtype=dtype)


def _adapt(name, T, n_in, n_out, rank, adapters, dtype, layout, ragged=False, pad=0, none=0.0):
    return dict(name=name, op="adapt", T=T, n_in=n_in, n_out=n_out, rank=rank, adapters=adapters, dtype=dtype,
                layout=layout, ragged=ragged, pad=pad, none=none)


def listed():
    return [
        # one token through a test-sized layer: nothing but latency
        _decode("token_tiny", T=1, H=256, E=16, K=2, I=128),
        # one token of one request, the production layer: ten experts' weights
        _decode("token", T=1, H=2560, E=512, K=10, I=1024),
        # the same with the narrower experts, the Q2_0 map and the shared expert
        _decode("token_shared_q2_0", T=1, H=2560, E=512, K=10, I=640, fmt="q2_0", shared=True),
        # a window of drafted tokens under verification, each with its request's adapter
        _decode("window_5_adapted", T=5, H=2560, E=512, K=10, I=1024, rank=16, adapters=8, dtype="bf16"),
        # a small model's batch: every expert gets many of the rows
        _decode("batch_33_few_experts", T=33, H=512, E=6, K=2, I=640, fmt="q2_0", shared=True),
        # the decode batch of a server: most hit experts get one row
        _decode("batch_32", T=32, H=2560, E=512, K=10, I=1024),
        # the largest batch, with hot experts (Zipf bias) and the shared expert on every row
        _decode("batch_64_shared_skewed", T=64, H=2560, E=512, K=10, I=640, fmt="q2_0", shared=True, skewed=True),
        # one token's adapter, the smallest call
        _adapt("adapter_token", T=1, n_in=2560, n_out=2560, rank=16, adapters=64, dtype="bf16", layout="tokens"),
        # a decode batch in which every request has an adapter of its own, ranks 1..64
        _adapt("adapter_batch_32", T=32, n_in=2560, n_out=2560, rank=64, adapters=32, dtype="fp16", layout="tokens",
               ragged=True),
        # odd sizes, padded rows, fp32 adapters, a third of the rows without one
        _adapt("adapter_odd_203", T=203, n_in=1000, n_out=333, rank=13, adapters=5, dtype="fp32", layout="prompts",
               pad=8, none=0.33),
        # prompts of several requests in one chunk
        _adapt("adapter_prompts_2k", T=2048, n_in=2560, n_out=2560, rank=16, adapters=16, dtype="bf16",
               layout="prompts", none=0.1),
        # the full prompt chunk with wide adapters
        _adapt("adapter_prompts_8k", T=8192, n_in=2560, n_out=2560, rank=64, adapters=16, dtype="bf16",
               layout="prompts", none=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges."""
    if rng.random() < 0.5:
        T = _log_int(rng, 1, 64)
        if rng.random() < 0.5:
            H, E, K, I = 2560, 512, 10, rng.choice([640, 1024])
        else:
            H, I = 128 * rng.randint(1, 16), 64 * rng.randint(1, 16)
            E = _log_int(rng, 2, 300)
            K = rng.randint(1, min(E, 12))
        adapters = rng.choice([0, 0, _log_int(rng, 1, 32)])
        c = _decode("", T, H, E, K, I, fmt=rng.choice(["q2_sym", "q2_0"]), shared=rng.random() < 0.4,
                    skewed=rng.random() < 0.3, rank=_log_int(rng, 1, 64) if adapters else 0, adapters=adapters,
                    dtype=rng.choice(["fp32", "fp16", "bf16"]))
        cap = max(work(x)["flops"] for x in listed() if x["op"] == "decode")
    else:
        wide = rng.random() < 0.5
        T = _log_int(rng, 1, 8192)
        n_in = 2560 if wide else _log_int(rng, 16, 2560)
        n_out = rng.choice([2560, 512]) if wide else _log_int(rng, 16, 2560)
        rank = rng.choice([8, 16, 32, 64]) if wide else _log_int(rng, 1, 96)
        c = _adapt("", T, n_in, n_out, rank, _log_int(rng, 1, 64), rng.choice(["fp32", "fp16", "bf16"]),
                   "tokens" if T <= 64 and rng.random() < 0.7 else "prompts", ragged=rng.random() < 0.4,
                   pad=rng.choice([0, 0, 4, 5]), none=rng.choice([0.0, 0.1, 0.5]))
        cap = max(work(x)["flops"] for x in listed() if x["op"] == "adapt")
    while work(c)["flops"] > cap:
        c["T"] = max(1, c["T"] // 2)
    del c["name"]
    return c


def _hit_experts(case):
    """How many routed experts T tokens are expected to hit: each token picks K
    of E evenly, or by its logits plus the Zipf bias."""
    T, E, K = case["T"], case["E"], case["K"]
    if not case["skewed"]:
        return E * (1.0 - (1.0 - K / E) ** T)
    rng = np.random.default_rng(0)
    logits = rng.normal(0.0, 0.05 * math.sqrt(case["H"]), (T, E)) - 2.4 * np.log(np.arange(1, E + 1))
    return float(len(np.unique(np.argsort(-logits, axis=1)[:, :K])))


def work(case):
    """Each weight, input and output once; the multiply-adds of the products."""
    T = case["T"]
    if case["op"] == "adapt":
        wb = torch.finfo(DTYPES[case["dtype"]]).bits // 8
        L, r, n_in, n_out = case["adapters"], case["rank"], case["n_in"], case["n_out"]
        with_one = T * (1.0 - case["none"])
        mean = r * (0.5 if case["ragged"] else 1.0)
        hit = L * (1.0 - (1.0 - 1.0 / L) ** with_one) if case["layout"] == "tokens" else min(L, with_one)
        return dict(bytes=hit * mean * (n_in + n_out) * wb + with_one * n_in * 4 + 2 * T * n_out * 4 + 4 * T,
                    flops=2.0 * with_one * mean * (n_in + n_out))
    H, E, K, I = case["H"], case["E"], case["K"], case["I"]
    hit = _hit_experts(case) + (1 if case["shared"] else 0)
    expert = 3 * H * I * (2 / 8 + 2 / BLOCK)
    b = hit * expert + 4.0 * H * E + 8.0 * T * H
    f = 2.0 * T * (K + (1 if case["shared"] else 0)) * 3 * H * I + 2.0 * T * H * E
    if case["adapters"]:
        wb = torch.finfo(DTYPES[case["dtype"]]).bits // 8
        L, r = case["adapters"], case["rank"]
        b += L * (1.0 - (1.0 - 1.0 / L) ** T) * r * 2 * H * wb
        f += 4.0 * T * r * H
    return dict(bytes=b, flops=f)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _hidden(T, H, g):
    """A normed hidden state: unit normal with a few outlier channels."""
    x = torch.randn((T, H), generator=g, device="cuda")
    hot = torch.randint(0, H, (max(1, H // 512),), generator=g, device="cuda")
    x[:, hot] *= 8.0
    return x


def _adapter_weights(L, r, n_in, n_out, dtype, ragged, g):
    a = (torch.randn((L, r, n_in), generator=g, device="cuda") / math.sqrt(n_in)).to(DTYPES[dtype])
    b = (torch.randn((L, n_out, r), generator=g, device="cuda") * 0.05).to(DTYPES[dtype])
    scale = torch.rand((L,), generator=g, device="cuda") * 1.5 + 0.5
    ranks = torch.randint(1, r + 1, (L,), generator=g, device="cuda", dtype=torch.int32) if ragged else None
    return a, b, scale, ranks


def _inputs_adapt(case, seed):
    g = _gen(seed)
    T, n_in, n_out, L, pad = case["T"], case["n_in"], case["n_out"], case["adapters"], case["pad"]
    x = _hidden(T, n_in + pad, g)[:, :n_in]
    y = torch.randn((T, n_out + pad), generator=g, device="cuda")[:, :n_out]
    a, b, scale, ranks = _adapter_weights(L, case["rank"], n_in, n_out, case["dtype"], case["ragged"], g)
    if case["layout"] == "tokens":  # a token of each of T requests
        ids = torch.randint(0, L, (T,), generator=g, device="cuda", dtype=torch.int32)
        drop = torch.rand((T,), generator=g, device="cuda") < case["none"]
        ids = torch.where(drop, torch.full_like(ids, -1), ids)
    else:  # prompts one after another, each of one request (some of a request without an adapter)
        n = min(T, max(L, 4))
        cuts = torch.sort(torch.randint(0, T, (n - 1,), generator=g, device="cuda")).values
        which = torch.randint(0, L, (n,), generator=g, device="cuda", dtype=torch.int32)
        drop = torch.rand((n,), generator=g, device="cuda") < case["none"]
        which = torch.where(drop, torch.full_like(which, -1), which)
        ids = which[torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)].contiguous()
    return dict(x=x, y=y, ids=ids, a=a, b=b, scale=scale, ranks=ranks)


def _inputs_decode(case, seed):
    g = _gen(seed)
    T, H, E, I = case["T"], case["H"], case["E"], case["I"]
    n = E + (1 if case["shared"] else 0)

    def codes(*shape):
        return torch.randint(0, 4, shape, generator=g, device="cuda", dtype=torch.uint8)

    def scales(*shape):
        return (torch.rand(shape, generator=g, device="cuda") * 0.015 + 0.005).to(torch.float16)

    s = dict(x=_hidden(T, H, g), router_w=torch.randn((H, E), generator=g, device="cuda") * 0.05,
             codes_gu=codes(n, 2 * I, H), scales_gu=scales(n, 2 * I, H // BLOCK),
             codes_d=codes(n, H, I), scales_d=scales(n, H, I // BLOCK), bias=None, shared_gate=None)
    if case["skewed"]:
        rank = torch.randperm(E, generator=g, device="cuda").double() + 1
        s["bias"] = (2.0 * torch.log(rank ** -1.2)).float()
    if case["shared"]:
        s["shared_gate"] = torch.randn((H,), generator=g, device="cuda") * 0.05
    if case["adapters"]:
        s["a"], s["b"], s["scale"], s["ranks"] = _adapter_weights(case["adapters"], case["rank"], H, H, case["dtype"],
                                                                  False, g)
        s["ids"] = torch.randint(0, case["adapters"], (T,), generator=g, device="cuda", dtype=torch.int32)
    return s


def _inputs(case, seed):
    return _inputs_adapt(case, seed) if case["op"] == "adapt" else _inputs_decode(case, seed)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import quantized_routed_expert_logits_amd as qm

    s["qm"] = qm
    if "a" in s:
        s["adapters"] = qm.Adapters(s["a"], s["b"], scale=s["scale"], ranks=s["ranks"])
    if case["op"] == "adapt":
        s["out"] = torch.empty((case["T"], case["n_out"]), device="cuda")
        nbytes = qm.strata_moe_adapt_workspace_bytes(case["T"], s["adapters"])
    else:
        ex = qm.Experts(case["E"], case["H"], case["I"], router_bias=s["bias"], device="cuda", fmt=case["fmt"],
                        shared=case["shared"])
        ex.pack(0, s.pop("codes_gu"), s.pop("scales_gu").view(torch.int16), s.pop("codes_d"),
                s.pop("scales_d").view(torch.int16))
        s["experts"] = ex.with_shared_gate(s["shared_gate"]) if case["shared"] else ex
        s["out"] = torch.empty_like(s["x"])
        nbytes = qm.strata_moe_decode_workspace_bytes(case["T"], case["K"], s["experts"], s.get("adapters"))
    s["workspace"] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------- run
def run(state):
    case = state["case"]
    if own:
        qm = state["qm"]
        if case["op"] == "adapt":
            return qm.strata_moe_adapt(state["x"], state["ids"], state["adapters"], state["y"], state["out"],
                                       workspace=state["workspace"])
        return qm.strata_moe_decode(state["x"], state["router_w"], state["experts"], case["K"], state["out"],
                                    adapters=state.get("adapters"), adapter_ids=state.get("ids"),
                                    workspace=state["workspace"])
    if case["op"] == "adapt":
        return _plain_adapt(state["x"], state["y"], state)
    y = _plain_decode(state, case)
    return _plain_adapt(state["x"], y, state) if case["adapters"] else y


def _plain_adapt(x, y, s):
    """out[t] = y[t] + scale B (A x[t]) with the weights of each token gathered."""
    a, b, ids = s["a"], s["b"], s["ids"].long()
    L, r = a.shape[0], a.shape[1]
    out = torch.empty((x.shape[0], b.shape[1]), device=x.device)
    step = max(1, (1 << 25) // max(a[0].numel(), b[0].numel()))
    for t0 in range(0, x.shape[0], step):
        at = ids[t0:t0 + step]
        one = (at >= 0) & (at < L)
        at = at.clamp(0, L - 1)
        v = torch.matmul(a[at].float(), x[t0:t0 + step].unsqueeze(-1)).squeeze(-1)
        if s["ranks"] is not None:
            v = torch.where(torch.arange(r, device=x.device) < s["ranks"][at].unsqueeze(-1), v, 0.0)
        d = torch.matmul(b[at].float(), v.unsqueeze(-1)).squeeze(-1) * s["scale"][at].unsqueeze(-1)
        yt = y[t0:t0 + step]
        out[t0:t0 + step] = torch.where(one.unsqueeze(-1), yt + d, yt)
    return out


def _round_int8(v):
    """Per 32 values: s = max|v| / 127 and q = round(v / s), halves away from
    zero, both divisions rounded to 32 bits (their operands are next to the
    borders that decide a code, hence the 64-bit quotients)."""
    blocks = v.reshape(*v.shape[:-1], -1, BLOCK)
    s = (blocks.abs().amax(-1).double() / 127.0).float()
    t = (blocks.double() / s.double().unsqueeze(-1)).float().double()
    q = torch.copysign(torch.floor(t.abs() + 0.5).clamp(max=127.0), t)
    q = torch.where(s.unsqueeze(-1) == 0, 0.0, q)
    return q.float(), s


def _block_rows(codes, scales, q, s, zero):
    """[T][M] = sum over blocks of scale s sum (code - zero) q; the sums within
    a block are exact in 32 bits, those over the blocks are in 64."""
    T, M = codes.shape[:2]
    p = ((codes.float() - zero).view(T, M, -1, BLOCK) * q.view(T, 1, -1, BLOCK)).sum(-1)
    return (p.double() * scales.double() * s.double().unsqueeze(1)).sum(-1)


def _plain_decode(s, case):
    zero, K, E = CODE_ZERO[case["fmt"]], case["K"], case["E"]
    x = s["x"]
    logits = x.double() @ s["router_w"].double()
    if s["bias"] is not None:
        logits = logits + s["bias"].double()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, w = ids[:, :K], torch.softmax(top[:, :K], dim=1)
    if case["shared"]:
        gate = torch.sigmoid(x.double() @ s["shared_gate"].double())
        ids = torch.cat([ids, torch.full_like(ids[:, :1], E)], 1)
        w = torch.cat([w, gate.unsqueeze(1)], 1)
    qx, sx = _round_int8(x)
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 25) // (2 * case["I"] * case["H"]))
    for t0 in range(0, x.shape[0], step):
        sl = slice(t0, t0 + step)
        for k in range(ids.shape[1]):
            e = ids[sl, k]
            gu = _block_rows(s["codes_gu"][e], s["scales_gu"][e], qx[sl], sx[sl], zero)
            gt, up = gu[:, :case["I"]], gu[:, case["I"]:]
            qh, sh = _round_int8((gt / (1.0 + torch.exp(-gt)) * up).float())
            out[sl] += w[sl, k:k + 1] * _block_rows(s["codes_d"][e], s["scales_d"][e], qh, sh, zero)
    return out.float()


# ------------------------------------------------------------------- exact
def exact(case, seed):
    s = _inputs(case, seed)
    x = s["x"].double()
    if case["op"] == "adapt":
        return _exact_adapt(x, s["y"].double(), s)
    y = _exact_layer(x, s, case)
    return _exact_adapt(x, y, s) if case["adapters"] else y


def _exact_adapt(x, y, s):
    """Adapter by adapter, on the rows that carry it."""
    out = y.clone()
    for a in range(s["a"].shape[0]):
        rows = (s["ids"] == a).nonzero().flatten()
        if rows.numel() == 0:
            continue
        r = s["a"].shape[1] if s["ranks"] is None else int(s["ranks"][a])
        down, up = s["a"][a, :r].double(), s["b"][a, :, :r].double()
        out[rows] += (x[rows] @ down.T) @ up.T * s["scale"][a].double()
    return out


def _exact_int8(v):
    """The values that the int8 rounding of the 32-bit rows v stands for."""
    blocks = v.float().double().unflatten(-1, (-1, BLOCK))
    top = blocks.abs().max(dim=-1, keepdim=True).values
    s = (top / 127.0).float().double()
    t = (blocks / torch.where(s > 0, s, 1.0)).float().double()
    q = torch.sign(t) * torch.floor(t.abs() + 0.5)
    return (q.clamp(-127.0, 127.0) * s).flatten(-2)


def _exact_weight(codes, scales, zero):
    return (codes.double() - zero) * scales.double().repeat_interleave(BLOCK, dim=-1)


def _exact_layer(x, s, case):
    """Expert by expert, on the rows routed to it, with dense 64-bit weights."""
    zero, K, E, I = CODE_ZERO[case["fmt"]], case["K"], case["E"], case["I"]
    logits = x @ s["router_w"].double() + (0.0 if s["bias"] is None else s["bias"].double())
    weight = torch.zeros((x.shape[0], E + 1), dtype=torch.float64, device=x.device)
    picked = torch.argsort(-logits, dim=1, stable=True)[:, :K]
    chosen = logits.gather(1, picked)
    e = torch.exp(chosen - chosen[:, :1])
    weight.scatter_(1, picked, e / e.sum(1, keepdim=True))
    hit = torch.zeros_like(weight, dtype=torch.bool).scatter_(1, picked, True)
    if case["shared"]:
        weight[:, E] = 1.0 / (1.0 + torch.exp(-(x @ s["shared_gate"].double())))
        hit[:, E] = True
    xi = _exact_int8(x)
    out = torch.zeros_like(x)
    for n in hit.any(0).nonzero().flatten().tolist():
        rows = hit[:, n].nonzero().flatten()
        gu = xi[rows] @ _exact_weight(s["codes_gu"][n], s["scales_gu"][n], zero).T
        h = gu[:, :I] / (1.0 + torch.exp(-gu[:, :I])) * gu[:, I:]
        d = _exact_int8(h) @ _exact_weight(s["codes_d"][n], s["scales_d"][n], zero).T
        out[rows] += weight[rows, n:n + 1] * d
    return out
