"""The workloads of the 4-bit floating-point products and of the norms around a block.

Four operators are run here, each over the range of sizes it is used at:

``quantize``  rows rounded to microscaled 4-bit floating point (a power of two
              per 32 values, 1-2-1 bit values), and the values that the codes
              stand for (``strata_moe_mxfp_quantize``, ``_dequantize``).
``product``   out[r] = W_e x[src[r]] for the rows r of each expert e, both sides
              in that format; with ``swiglu`` the rows of W are [gate; up] and
              out[r] = silu(g) u (``strata_moe_mxfp_product``).  With one expert
              and no grouping it is a plain projection.
``before``    the layer's input from the residual stream: x = norm(h), a root
              mean square norm (``strata_moe_norm_before``).
``after``     the layer's output into the residual stream: the weighted sum of a
              token's K expert rows, its norm, gate and scales, the addition to
              the stream, and the norm (and 4-bit rounding) that the next block
              reads (``strata_moe_norm_after``).

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from
a seed, ``run`` is one call.  With ``own`` false the call is spelled out in
elementary torch operations; with ``own`` true it goes through the library.
``exact`` evaluates the definition in 64 bits.
"""
import math

import torch

own = False

BLOCK = 32
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def _quantize(name, T, H, dtype, pad=0):
    return dict(name=name, op="quantize", T=T, H=H, dtype=dtype, pad=pad)


def _product(name, T, n_in, n_out, E=1, K=1, swiglu=False, skewed=False, gather=True, dtype="fp32", pad=0):
    """n_out: the outputs of one row (with swiglu the weights have twice as many rows).  E = 1: no grouping."""
    return dict(name=name, op="product", T=T, n_in=n_in, n_out=n_out, E=E, K=K, swiglu=swiglu, skewed=skewed,
                gather=gather, dtype=dtype, pad=pad)


def _before(name, T, H, dtype, codes=False, pad=0, offset=0.0):
    return dict(name=name, op="before", T=T, H=H, dtype=dtype, codes=codes, pad=pad, offset=offset)


def _after(name, T, H, dtype, K=0, y_dtype="fp32", norm=True, gate="none", follow=False, codes=False, pad=0):
    return dict(name=name, op="after", T=T, H=H, dtype=dtype, K=K, y_dtype=y_dtype, norm=norm, gate=gate,
                follow=follow, codes=codes, pad=pad)


def listed():
    return [
        # a short prompt of odd width out of a wider array
        _quantize("quantize_odd_203", T=203, H=1056, dtype="bf16", pad=8),
        # the layer input of a full prompt chunk
        _quantize("quantize_8k", T=8192, H=2560, dtype="fp32"),
        # one token's ten experts, gate/up of the production layer
        _product("gate_up_token", T=1, n_in=2560, n_out=1024, E=512, K=10, swiglu=True),
        # the decode batch of a server: most hit experts get one row
        _product("down_batch_32", T=32, n_in=1024, n_out=2560, E=512, K=10, gather=False),
        # few experts, a reduction that ends inside a step, an odd number of outputs, padded rows
        _product("experts_odd_203", T=203, n_in=544, n_out=333, E=6, K=2, dtype="fp16", pad=3),
        # the full prompt chunk: gate/up, hot experts among the 512
        _product("gate_up_8k", T=8192, n_in=2560, n_out=1024, E=512, K=10, swiglu=True, skewed=True, dtype="bf16"),
        # and down
        _product("down_8k", T=8192, n_in=1024, n_out=2560, E=512, K=10, gather=False, dtype="bf16"),
        # a projection that every token takes, at the widest layer
        _product("projection_8k", T=8192, n_in=4096, n_out=4096, dtype="bf16"),
        # one token's norm before the layer: latency alone
        _before("before_token", T=1, H=2560, dtype="bf16"),
        # a prompt chunk of odd width, weights stored around zero
        _before("before_odd_2k", T=2047, H=1001, dtype="fp32", pad=3, offset=1.0),
        # the decode batch: ten expert rows a token, a channel gate, the next block's norm
        _after("after_batch_32", T=32, H=2560, dtype="bf16", K=10, gate="channel", follow=True),
        # the full prompt chunk, with the next block's input rounded to 4 bits
        _after("after_8k", T=8192, H=2560, dtype="bf16", K=10, y_dtype="bf16", gate="token", follow=True, codes=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["quantize", "product", "product", "before", "after"])
    T = _log_int(rng, 1, 8192)
    dtype = rng.choice(["fp32", "fp16", "bf16"])
    pad = rng.choice([0, 0, 0, 1, 8])
    wide = rng.random() < 0.4
    if op == "quantize":
        c = _quantize("", T, 2560 if wide else BLOCK * _log_int(rng, 1, 128), dtype, pad)
    elif op == "product":
        form = rng.choice(["experts", "experts", "small", "dense"])
        if form == "experts":
            E, K, n_in, n_out = 512, 10, 2560, rng.choice([640, 1024])
            swiglu = rng.random() < 0.5
            if not swiglu:
                n_in, n_out = n_out, n_in
        else:
            E = _log_int(rng, 2, 300) if form == "small" else 1
            K = rng.randint(1, min(E, 12))
            n_in, n_out = BLOCK * _log_int(rng, 1, 128), _log_int(rng, 1, 4096)
            swiglu = rng.random() < 0.3
        c = _product("", T, n_in, n_out, E, K, swiglu=swiglu, skewed=rng.random() < 0.3, gather=rng.random() < 0.5,
                     dtype=dtype, pad=pad)
    elif op == "before":
        c = _before("", T, 2560 if wide else _log_int(rng, 1, 4096), dtype, pad=pad, offset=rng.choice([0.0, 1.0]))
        if c["H"] % BLOCK == 0:
            c["codes"] = rng.random() < 0.4
    else:
        c = _after("", T, 2560 if wide else _log_int(rng, 1, 4096), dtype, K=rng.choice([0, 1, 4, 10]),
                   y_dtype=rng.choice(["fp32", "fp16", "bf16"]), norm=rng.random() < 0.7,
                   gate=rng.choice(["none", "channel", "token", "full"]), follow=rng.random() < 0.6, pad=pad)
        if c["follow"] and c["H"] % BLOCK == 0:
            c["codes"] = rng.random() < 0.4
    caps = [work(x) for x in listed() if x["op"] == op]
    while any(work(c)[k] > max(x[k] for x in caps) for k in ("bytes", "flops")):
        c["T"] = max(1, c["T"] // 2)
        if c["T"] == 1:
            break
    del c["name"]
    return c


def _size(dtype):
    return torch.finfo(DTYPES[dtype]).bits // 8


PACKED = 0.5 + 1.0 / BLOCK  # bytes of a 4-bit value with its share of the scale


def work(case):
    """Each weight, input and output once; the multiply-adds of the products."""
    T = case["T"]
    if case["op"] == "product":
        n_in, n_out, E, K = case["n_in"], case["n_out"], case["E"], case["K"]
        n_w = n_out * (2 if case["swiglu"] else 1)
        if E == 1:
            hit, rows = 1, T
        else:
            share = _shares(E, case["skewed"])
            hit, rows = sum(1.0 - (1.0 - min(1.0, K * p)) ** T for p in share), T * K
        x_rows = T if E == 1 or case["gather"] else rows
        b = hit * n_w * n_in * PACKED + x_rows * n_in * PACKED + rows * n_out * _size(case["dtype"])
        return dict(bytes=b + (4.0 * (rows if case["gather"] else 0) + 4.0 * E if E > 1 else 0),
                    flops=2.0 * rows * n_w * n_in)
    H = case["H"]
    n = T * H
    if case["op"] == "quantize":  # in, codes out and in again, values out
        return dict(bytes=n * (2.0 * _size(case["dtype"]) + 2.0 * PACKED), flops=4.0 * n)
    coded = (2.0 * PACKED + 4.0) * n if case["codes"] else 0.0
    if case["op"] == "before":
        return dict(bytes=n * (_size(case["dtype"]) + 4.0) + 4.0 * H + coded, flops=4.0 * n)
    K = case["K"]
    b = n * 2.0 * _size(case["dtype"]) + n * max(K, 1) * _size(case["y_dtype"]) + 8.0 * T * K
    b += {"none": 0.0, "channel": 4.0 * H, "token": 4.0 * T, "full": 4.0 * n}[case["gate"]]
    b += (4.0 * H if case["norm"] else 0.0) + ((4.0 * n + 4.0 * H) if case["follow"] else 0.0) + coded
    return dict(bytes=b, flops=n * (2.0 * max(K, 1) + 8.0))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _shares(E, skewed):
    """How often a router picks each expert, relative to all picks."""
    w = [1.0 / (i + 8.0) if skewed else 1.0 for i in range(E)]
    return [v / sum(w) for v in w]


def _hidden(T, H, g):
    """A hidden state: unit normal with a few outlier channels."""
    x = torch.randn((T, H), generator=g, device="cuda")
    hot = torch.randint(0, H, (max(1, H // 512),), generator=g, device="cuda")
    x[:, hot] *= 8.0
    return x


def _pick(T, E, K, skewed, g):
    """K experts for each of T tokens (none twice), grouped: (offsets [E+1],
    src [T K] the token of each grouped row, slot [T K] the row of each pair)."""
    share = torch.tensor(_shares(E, skewed), device="cuda").log()
    share = share[torch.randperm(E, generator=g, device="cuda")]
    noise = torch.rand((T, E), generator=g, device="cuda").clamp(min=1e-9)
    ids = torch.topk(share - torch.log(-torch.log(noise)), K, dim=1).indices.flatten()
    order = torch.sort(ids, stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(ids, minlength=E), 0).int()
    slot = torch.empty_like(order)
    slot[order] = torch.arange(T * K, device="cuda")
    return offsets, (order // K).int(), slot.int()


def _packed(codes):
    """Codes 0..15 -> two to a byte, the first in the low half."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _split(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def _inputs_product(case, g):
    T, n_in, n_out, E, K = case["T"], case["n_in"], case["n_out"], case["E"], case["K"]
    n_w = n_out * (2 if case["swiglu"] else 1)
    s = dict(offsets=None, src=None)
    x_rows = rows = T
    if E > 1:
        rows = T * K
        s["offsets"], src, _ = _pick(T, E, K, case["skewed"], g)
        if case["gather"]:
            s["src"] = src
        else:
            x_rows = rows
    s["rows"] = rows
    codes, scales = _round_mxfp(_hidden(x_rows, n_in, g))
    s["x_codes"], s["x_scales"] = _packed(codes), scales
    # weights as a 4-bit pack holds them: every code about as often, scales a few powers of two around 2^-8
    s["w_codes"] = torch.randint(0, 256, (E, n_w, n_in // 2), generator=g, device="cuda", dtype=torch.uint8)
    s["w_scales"] = torch.randint(117, 121, (E, n_w, n_in // BLOCK), generator=g, device="cuda", dtype=torch.uint8)
    return s


def _norm_weight(H, offset, g):
    return 1.0 - offset + 0.2 * torch.randn((H,), generator=g, device="cuda")


def _inputs(case, seed):
    g = _gen(seed)
    if case["op"] == "product":
        return _inputs_product(case, g)
    T, H, pad, dt = case["T"], case["H"], case["pad"], DTYPES[case["dtype"]]
    if case["op"] == "quantize":
        return dict(x=_hidden(T, H + pad, g).to(dt)[:, :H])
    s = dict(h=(3.0 * _hidden(T, H + pad, g)).to(dt)[:, :H])
    if case["op"] == "before":
        s["weight"] = _norm_weight(H, case["offset"], g)
        return s
    K = case["K"]
    s["y"] = torch.randn((T * max(K, 1), H), generator=g, device="cuda").to(DTYPES[case["y_dtype"]])
    s["slot"] = s["p"] = s["gate"] = s["weight"] = s["next"] = None
    if K:
        s["slot"] = torch.randperm(T * K, generator=g, device="cuda").int().view(T, K)
        s["p"] = torch.softmax(torch.randn((T, K), generator=g, device="cuda"), 1)
    if case["gate"] != "none":
        shape = {"channel": (H,), "token": (T, 1), "full": (T, H)}[case["gate"]]
        s["gate"] = torch.sigmoid(torch.randn(shape, generator=g, device="cuda"))
    if case["norm"]:
        s["weight"] = _norm_weight(H, 0.0, g)
    if case["follow"]:
        s["next"] = _norm_weight(H, 0.0, g)
    return s


RESIDUAL_SCALE, BLOCK_SCALE = 1.0, 0.75


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import quantized_routed_expert_logits_amd as qm

    s["qm"] = qm
    T, dt = case["T"], DTYPES[case["dtype"]]

    def empty(rows, cols, dtype, pad=0):
        return torch.empty((rows, cols + pad), dtype=dtype, device="cuda")[:, :cols]

    if case["op"] == "product":
        w = qm.MxfpWeights(case["E"], s["w_codes"].shape[1], case["n_in"], swiglu=case["swiglu"], device="cuda")
        w.pack(0, s.pop("w_codes"), s.pop("w_scales"))
        s["weights"] = w
        s["out"] = empty(s["rows"], case["n_out"], dt, case["pad"])
        return s
    H = case["H"]
    if case["op"] == "quantize":
        s["out"] = empty(T, H, dt)
    if case["op"] == "after":
        s["out"] = empty(T, H, dt, case["pad"])
        s["norm"] = None if s["weight"] is None else qm.Norm(s["weight"], eps=EPS)
        s["next_norm"] = None if s["next"] is None else qm.Norm(s["next"], eps=EPS)
    if case["op"] == "before":
        s["norm"] = qm.Norm(s["weight"], eps=EPS, weight_offset=case["offset"])
    s["x_out"] = torch.empty((T, H), device="cuda") if case["op"] == "before" or case.get("follow") else None
    coded = case["op"] == "quantize" or case["codes"]
    s["codes"] = torch.empty((T, H // 2), dtype=torch.uint8, device="cuda") if coded else None
    s["scales"] = torch.empty((T, H // BLOCK), dtype=torch.uint8, device="cuda") if coded else None
    s["values"] = torch.empty((T, H), device="cuda") if coded and case["op"] != "quantize" else None
    return s


# --------------------------------------------------------------------- run
def run(state):
    case = state["case"]
    return _run_own(state, case) if own else _run_plain(state, case)


def _run_own(s, case):
    qm = s["qm"]
    if case["op"] == "quantize":
        codes, scales = qm.strata_moe_mxfp_quantize(s["x"], s["codes"], s["scales"])
        return qm.strata_moe_mxfp_dequantize(codes, scales, s["out"])
    if case["op"] == "product":
        return qm.strata_moe_mxfp_product(s["x_codes"], s["x_scales"], s["weights"], s["out"], offsets=s["offsets"],
                                         src=s["src"])
    if case["op"] == "before":
        qm.strata_moe_norm_before(s["h"], s["norm"], s["x_out"], codes=s["codes"], scales=s["scales"])
        res = [s["x_out"]]
    else:
        qm.strata_moe_norm_after(s["h"], s["y"], s["out"], norm=s["norm"], slot=s["slot"], p=s["p"], gate=s["gate"],
                                 residual_scale=RESIDUAL_SCALE, block_scale=BLOCK_SCALE, next_norm=s["next_norm"],
                                 x=s["x_out"], codes=s["codes"], scales=s["scales"])
        res = [s["out"]] + ([s["x_out"]] if case["follow"] else [])
    if case["codes"]:
        res.append(qm.strata_moe_mxfp_dequantize(s["codes"], s["scales"], s["values"]))
    return res


def _power(byte):
    """2^(byte - 127) in 32 bits, NaN for 255."""
    return torch.where(byte == 255, math.nan, torch.ldexp(torch.ones((), device=byte.device), byte.int() - 127))


def _round_mxfp(x):
    """[..., n] -> codes 0..15 [..., n] and scale bytes [..., n / 32]: a power
    of two 2^e with e = floor(log2(largest magnitude)) - 2, and each value over
    it rounded to the nearest of the eight magnitudes (ties to the even code,
    larger ones to 6)."""
    v = x.float().unflatten(-1, (-1, BLOCK))
    top = v.abs().amax(-1)
    e = (torch.frexp(top).exponent - 3).clamp(-127, 127)
    e = torch.where(top == 0, -127, e)
    q = torch.ldexp(v, -e.unsqueeze(-1)).abs()
    mids = [(a + b) / 2 for a, b in zip(MAGNITUDES, MAGNITUDES[1:])]
    code = torch.zeros(q.shape, dtype=torch.uint8, device=x.device)
    for i, m in enumerate(mids):
        code += ((q >= m) if i % 2 else (q > m)).to(torch.uint8)
    code |= torch.signbit(v).to(torch.uint8) << 3
    return code.flatten(-2), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """What codes 0..15 and their scale bytes stand for, in 32 bits."""
    m = torch.tensor(MAGNITUDES, device=codes.device)
    table = torch.cat([m, -m])
    v = table[codes.int()].unflatten(-1, (-1, BLOCK)) * _power(scales).unsqueeze(-1)
    return v.flatten(-2)


def _run_plain(s, case):
    if case["op"] == "quantize":
        return _values(*_round_mxfp(s["x"])).to(s["x"].dtype)
    if case["op"] == "product":
        return _plain_product(s, case)
    if case["op"] == "before":
        x = _plain_norm(s["h"].double(), s["weight"], case["offset"]).float()
        return [x] + ([_values(*_round_mxfp(x))] if case["codes"] else [])
    return _plain_after(s, case)


def _plain_norm(v, weight, offset):
    """In 64 bits: the 4-bit rounding that may follow has values next to its borders."""
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * (offset + weight.double())


def _plain_after(s, case):
    y = s["y"].double()
    if case["K"]:
        y = (y[s["slot"].long()] * s["p"].double().unsqueeze(-1)).sum(1)
    if case["norm"]:
        y = _plain_norm(y, s["weight"], 0.0)
    if s["gate"] is not None:
        y = y * s["gate"].double()
    out = (RESIDUAL_SCALE * s["h"].double() + BLOCK_SCALE * y).to(s["h"].dtype)
    res = [out]
    if case["follow"]:
        res.append(_plain_norm(out.double(), s["next"], 0.0).float())
        if case["codes"]:
            res.append(_values(*_round_mxfp(res[1])))
    return res


def _plain_product(s, case):
    dt = DTYPES[case["dtype"]]
    x = _values(_split(s["x_codes"]), s["x_scales"])
    if s["src"] is not None:
        x = x[s["src"].long()]
    out = torch.empty((s["rows"], case["n_out"]), dtype=dt, device=x.device)
    cuts = [0, s["rows"]] if s["offsets"] is None else s["offsets"].tolist()
    for e, (r0, r1) in enumerate(zip(cuts, cuts[1:])):
        if r1 == r0:
            continue
        y = x[r0:r1] @ _values(_split(s["w_codes"][e]), s["w_scales"][e]).T
        if case["swiglu"]:
            gate, up = y[:, :case["n_out"]], y[:, case["n_out"]:]
            y = gate / (1.0 + torch.exp(-gate)) * up
        out[r0:r1] = y.to(dt)
    return out


# ------------------------------------------------------------------- exact
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "quantize":
        return _exact_mxfp(s["x"].double())
    if case["op"] == "product":
        return _exact_product(s, case)
    if case["op"] == "before":
        x = _exact_norm(s["h"].double(), s["weight"].double() + case["offset"])
        return [x] + ([_exact_mxfp(x.float().double())] if case["codes"] else [])
    return _exact_after(s, case)


def _exact_mxfp(x):
    """The values that the 4-bit rounding of x stands for: on the grid of step
    max(2^(floor(log2|q|) - 1), 1/2) below 6, halves to the even multiple."""
    v = x.unflatten(-1, (-1, BLOCK))
    top = v.abs().amax(-1, keepdim=True)
    unit = torch.exp2(torch.floor(torch.log2(top) + 1e-12) - 2.0).clamp(min=2.0 ** -127, max=2.0 ** 127)
    q = v / unit
    step = torch.where(q.abs() >= 4.0, 2.0, torch.where(q.abs() >= 2.0, 1.0, 0.5))
    q = (torch.round(q / step) * step).clamp(-6.0, 6.0)
    return torch.where(top == 0, 0.0, q * unit).flatten(-2)


def _exact_values(packed, scales):
    """Sign, exponent and mantissa bits read one by one."""
    c = torch.stack([torch.bitwise_and(packed, 15), torch.bitwise_right_shift(packed, 4)], dim=-1)
    c = c.reshape(*packed.shape[:-1], -1).to(torch.int16)
    expo, man = ((c >> 1) & 3).double(), (c & 1).double()
    mag = torch.where(expo == 0, 0.5 * man, torch.exp2(expo - 1.0) * (1.0 + 0.5 * man))
    unit = torch.exp2(scales.double() - 127.0).repeat_interleave(BLOCK, dim=-1)
    return torch.where(c >= 8, -mag, mag) * unit


def _exact_product(s, case):
    x = _exact_values(s["x_codes"], s["x_scales"])
    out = torch.zeros((s["rows"], case["n_out"]), dtype=torch.float64, device=x.device)
    for e in range(case["E"]):
        lo, hi = (0, s["rows"]) if s["offsets"] is None else (int(s["offsets"][e]), int(s["offsets"][e + 1]))
        if lo == hi:
            continue
        rows = torch.arange(lo, hi, device=x.device)
        if s["src"] is not None:
            rows = s["src"][lo:hi].long()
        y = torch.matmul(_exact_values(s["w_codes"][e], s["w_scales"][e]), x[rows].T).T
        if case["swiglu"]:
            g, u = torch.chunk(y, 2, dim=1)
            y = g * u * torch.sigmoid(g)
        out[lo:hi] = y
    return out


def _exact_norm(v, scale):
    return scale * v * torch.rsqrt(v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS)


def _exact_after(s, case):
    h, y = s["h"].double(), s["y"].double()
    if case["K"]:
        v = torch.zeros_like(h)
        for k in range(case["K"]):
            v += s["p"][:, k:k + 1].double() * y[s["slot"][:, k].long()]
        y = v
    if case["norm"]:
        y = _exact_norm(y, s["weight"].double())
    gate = 1.0 if s["gate"] is None else s["gate"].double()
    out = h * RESIDUAL_SCALE + y * gate * BLOCK_SCALE
    res = [out]
    if case["follow"]:  # the next block reads the stream as it is stored
        x = _exact_norm(out.to(s["h"].dtype).double(), s["next"].double())
        res.append(x)
        if case["codes"]:
            res.append(_exact_mxfp(x.float().double()))
    return res
