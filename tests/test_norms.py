"""The norms around a block (strata_moe_norm_before, _after) against their
definition in 64 bits.

Tolerance: the kernels work in fp64 and round an output to fp32, and from there
to a 16-bit type.  Their sums have at most H + K + 40 roundings of 2^-53 relative
to the absolute terms (H <= 16384), below 2^-38, so an output is off by half a
step of its type, half a step of fp32 and 2^-37 of the absolute terms.  The
stream that the next norm reads is the stored one.
4-bit codes: those of the fp32 x that the same call wrote, bit for bit.
"""
import ctypes

import mxfp_reference as ref
import numpy as np
import pytest
import torch

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
IDS = ["fp32", "fp16", "bf16"]
SMALL = 2.0 ** -37


@pytest.fixture(scope="module")
def qm():
    import quantized_routed_expert_logits_amd as qm
    return qm


def _np(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _close(got, want, terms):
    dt = torch.finfo(got.dtype)
    tol = ref.rounding(dt.eps, dt.smallest_normal * dt.eps, np.abs(want)) + 2.0 ** -24 * np.abs(want) + SMALL * terms
    err = np.abs(_np(got) - want)
    assert np.all(err <= tol), f"worst {np.nanmax(err / tol):.3f} of the tolerance"


def _check_codes(x, codes, scales):
    c, b = ref.quantize(_np(x))
    assert np.array_equal(_np(scales), b) and np.array_equal(_np(codes), ref.pack(c))


def _rows(T, H, pad, dtype, g, scale=1.0):
    return (torch.randn((T, H + pad), generator=g) * scale).to(dtype).cuda()[:, :H]


BEFORE = [(1, 1, 0), (1, 2560, 0), (2, 3, 1), (5, 33, 0), (7, 64, 1), (33, 255, 2), (64, 256, 8), (100, 1001, 3),
          (40, 2560, 0), (3, 4096, 4), (3, 4100, 0), (2, 8192, 1), (2, 16384, 0), (2, 12001, 0), (1025, 96, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("size", BEFORE, ids=lambda s: "-".join(map(str, s)))
def test_before(qm, size, dtype):
    T, H, pad = size
    g = torch.Generator().manual_seed(T + H)
    h = _rows(T, H, pad, dtype, g, 3.0)
    w = torch.randn(H, generator=g).cuda()
    for weight, offset, eps in ((w, 0.0, 1e-6), (w, 1.0, 1e-5), (None, 0.0, 0.0),
                                (w[:0].new_ones(H + 1)[1:], 0.0, 0.5)):
        x = torch.empty((T, H), device="cuda")
        codes = scales = None
        if H % 32 == 0:
            codes = torch.empty((T, H // 2), dtype=torch.uint8, device="cuda")
            scales = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
        qm.strata_moe_norm_before(h, qm.Norm(weight, eps, offset), x, codes, scales)
        want = ref.norm(_np(h), None if weight is None else _np(weight), offset, eps)
        _close(x, want, np.abs(want))
        if codes is not None:
            _check_codes(x, codes, scales)
            c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
            qm.strata_moe_norm_before(h, qm.Norm(weight, eps, offset), codes=c2, scales=s2)  # codes alone
            assert torch.equal(codes, c2) and torch.equal(scales, s2)


AFTER = [  # T, H, pad, K, y dtype, gate, norm, next
    (1, 1, 0, 0, 0, "none", True, True), (1, 2560, 0, 10, 0, "channel", True, True),
    (3, 64, 1, 0, 1, "token", False, True), (7, 33, 0, 1, 2, "full", True, False),
    (32, 2560, 0, 10, 2, "token", True, True), (65, 1001, 3, 4, 1, "channel", True, True),
    (200, 96, 0, 16, 0, "full", False, True), (4, 4100, 0, 3, 2, "none", True, True),
    (2, 16384, 0, 2, 0, "token", True, True), (500, 256, 8, 0, 2, "none", True, True),
    (9, 640, 2, 2, 1, "wide", True, True),
]


def _after_case(T, H, pad, K, ydt, gate, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    s = dict(h=_rows(T, H, pad, dtype, g, 2.0), y=_rows(T * max(K, 1), H, pad, DTYPES[ydt], g), slot=None, p=None,
             gate=None)
    if K:
        s["slot"] = torch.randperm(T * K, generator=g).int().view(T, K).cuda()
        s["p"] = torch.rand((T, K), generator=g).cuda()
    if gate == "wide":  # rows of a wider array
        s["gate"] = torch.rand((T, H + 3), generator=g).cuda()[:, :H]
    elif gate != "none":
        s["gate"] = torch.rand({"channel": (H,), "token": (T, 1), "full": (T, H)}[gate], generator=g).cuda()
    return s, torch.randn(H, generator=g).cuda(), torch.randn(H, generator=g).cuda()


def _after_reference(s, weight, rs, bs, eps):
    """(out in 64 bits, absolute terms)."""
    h, y = _np(s["h"]), _np(s["y"])
    if s["slot"] is not None:
        slot, p = _np(s["slot"]), _np(s["p"])
        ok = (slot >= 0) & (slot < len(y))
        rows = y[np.clip(slot, 0, len(y) - 1)]
        pk = np.where(ok, p, 0.0)[..., None]
        v, mag = (pk * np.where(ok[..., None], rows, 0.0)).sum(1), (np.abs(pk) * np.abs(rows)).sum(1)
    else:
        v, mag = y, np.abs(y)
    gate = 1.0 if s["gate"] is None else _np(s["gate"])
    if weight is None:
        b = v
    else:
        b = ref.norm(v, _np(weight), 0.0, eps)
        r = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
        mag = mag * r * np.abs(_np(weight)) + np.abs(b)
    return rs * h + bs * (gate * b), np.abs(rs * h) + np.abs(bs * gate) * mag


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("size", AFTER, ids=lambda s: "-".join(map(str, s)))
def test_after(qm, size, dtype):
    T, H, pad, K, ydt, gate, with_norm, follow = size
    s, w, u = _after_case(T, H, pad, K, ydt, gate, dtype, seed=T + H)
    rs, bs, eps = 1.25, 0.3, 1e-6
    buf = torch.full((T, H + 5), 7.0, dtype=dtype, device="cuda")
    out = buf[:, :H]
    x = torch.empty((T, H), device="cuda") if follow else None
    codes = scales = None
    if follow and H % 32 == 0:
        codes = torch.empty((T, H // 2), dtype=torch.uint8, device="cuda")
        scales = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
    kw = dict(norm=qm.Norm(w, eps) if with_norm else None, slot=s["slot"], p=s["p"], gate=s["gate"], residual_scale=rs,
              block_scale=bs, next_norm=qm.Norm(u, eps, 1.0) if follow else None, x=x, codes=codes, scales=scales)
    qm.strata_moe_norm_after(s["h"], s["y"], out, **kw)
    want, terms = _after_reference(s, w if with_norm else None, rs, bs, eps)
    _close(out, want, terms)
    assert torch.all(buf[:, H:] == 7.0)
    if follow:
        xw = ref.norm(_np(out), _np(u), 1.0, eps)
        _close(x, xw, np.abs(xw))
        # as the norm alone gives it from the stored stream
        alone = torch.empty_like(x)
        qm.strata_moe_norm_before(out, qm.Norm(u, eps, 1.0), alone)
        assert torch.equal(alone, x)
    if codes is not None:
        _check_codes(x, codes, scales)
    # in place
    h2 = s["h"].clone()
    qm.strata_moe_norm_after(h2, s["y"], h2, **kw)
    assert torch.equal(h2, out)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES[1:], ids=IDS[1:])
def test_rounded_as_a_tensor_is(qm, dtype):
    """The stored stream is the 64-bit sum as torch makes a 16-bit tensor of it, bit for bit,
    at sums on and next to the middle of two values, subnormal ones and overflow."""
    g = torch.Generator().manual_seed(4)
    h = torch.randn((64, 512), generator=g).to(dtype)
    h[:8] *= 2.0 ** -13
    ulp = torch.finfo(dtype).eps * 2.0 ** torch.floor(torch.log2(h.float().abs().clamp(min=1e-6)))
    a = ulp / 2 * torch.randint(-1, 2, h.shape, generator=g)
    b = ulp * 2.0 ** -torch.randint(20, 34, h.shape, generator=g).float() * torch.randint(-1, 2, h.shape, generator=g)
    h[8], a[8] = torch.finfo(dtype).max, torch.finfo(dtype).max * torch.rand(512, generator=g)
    rows = torch.stack([a, b], 1).view(128, 512).cuda()  # y = a + b exactly, as two rows of weight 1
    slot = torch.arange(128, dtype=torch.int32).view(64, 2).cuda()
    out = torch.empty_like(h, device="cuda")
    qm.strata_moe_norm_after(h.cuda(), rows, out, slot=slot, p=torch.ones((64, 2)).cuda())
    assert torch.equal(out.cpu(), (h.double() + a.double() + b.double()).to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_extremes(qm, dtype):
    H = 96
    h = torch.randn((6, H), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    h[0] = 0.0
    h[1, 5] = float("nan")
    h[2, 7] = float("inf")
    h[3] = torch.finfo(dtype).max
    h[4] = torch.finfo(dtype).smallest_normal
    x = torch.empty((6, H), device="cuda")
    codes = torch.empty((6, 48), dtype=torch.uint8, device="cuda")
    scales = torch.empty((6, 3), dtype=torch.uint8, device="cuda")
    qm.strata_moe_norm_before(h, qm.Norm(None, 1e-12), x, codes, scales)
    assert torch.all(x[0] == 0) and torch.isnan(x[1]).all()
    # an infinite value: 0 where the others are finite, NaN at its own place
    assert torch.isnan(x[2, 7]) and torch.all(x[2, :7] == 0) and torch.all(x[2, 8:] == 0)
    want = ref.norm(_np(h[3:]), None, 0.0, 1e-12)
    _close(x[3:], want, np.abs(want))
    _check_codes(x, codes, scales)
    # no epsilon and a row of zeros: 0 / 0
    qm.strata_moe_norm_before(h[:1], qm.Norm(None, 0.0), x[:1])
    assert torch.isnan(x[0]).all()


@pytest.mark.gpu
def test_slots_outside_add_nothing(qm):
    T, H, K = 9, 130, 3
    s, w, _ = _after_case(T, H, 0, K, 0, "none", torch.float32, 5)
    s["slot"][0, 0], s["slot"][1, 2], s["slot"][2, 1] = -1, T * K, 2 ** 31 - 1
    s["slot"][3] = -2 ** 31
    out = torch.empty_like(s["h"])
    qm.strata_moe_norm_after(s["h"], s["y"], out, norm=qm.Norm(w, 1e-6), slot=s["slot"], p=s["p"])
    want, terms = _after_reference(s, w, 1.0, 1.0, 1e-6)
    _close(out, want, terms)
    assert torch.equal(out[3], s["h"][3])


@pytest.mark.gpu
def test_columns_of_one_array_and_repeats(qm):
    """h and out as columns of one array; the same bits again; rows behind T left."""
    T, H = 37, 320
    buf = torch.randn((T + 4, 2 * H + 7), generator=torch.Generator().manual_seed(2)).cuda()
    keep = buf.clone()
    h, out = buf[:T, :H], buf[:T, H:2 * H]
    y = torch.randn((T, H), generator=torch.Generator().manual_seed(3)).cuda()
    qm.strata_moe_norm_after(h, y, out, norm=qm.Norm(None, 1e-6))
    first = out.clone()
    qm.strata_moe_norm_after(h, y, out, norm=qm.Norm(None, 1e-6))
    assert torch.equal(first, out)
    keep[:T, H:2 * H] = first
    assert torch.equal(keep, buf)
    want, terms = _after_reference(dict(h=h, y=y, slot=None, gate=None), torch.ones(H), 1.0, 1.0, 1e-6)
    _close(out, want, terms)


def _layer(qm, s):
    """One block with 4-bit experts on the stream s["h"], in place."""
    qm.strata_moe_norm_before(s["h"], s["n1"], s["x"], s["xc"], s["xs"])
    qm.strata_moe_mxfp_product(s["xc"], s["xs"], s["gate_up"], s["hid"], offsets=s["offsets"], src=s["src"])
    qm.strata_moe_mxfp_quantize(s["hid"], s["hc"], s["hs"])
    qm.strata_moe_mxfp_product(s["hc"], s["hs"], s["down"], s["y"], offsets=s["offsets"])
    qm.strata_moe_norm_after(s["h"], s["y"], s["h"], norm=s["n2"], slot=s["slot"], p=s["p"], block_scale=0.5,
                             next_norm=s["n3"], x=s["x2"], codes=s["xc"], scales=s["xs"])


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,E,K", [(1, 256, 96, 16, 2), (50, 320, 160, 24, 4), (700, 256, 128, 8, 3)])
def test_a_block_with_4_bit_experts(qm, T, H, I, E, K):
    """Norm, route, group, gate/up, rounding, down, combine and the next norm, each
    step against its definition on the step before it; then captured and replayed."""
    g = torch.Generator().manual_seed(T)
    rnd = lambda *a: torch.randn(a, generator=g).cuda()  # noqa: E731
    u8 = lambda *a: torch.empty(a, dtype=torch.uint8, device="cuda")  # noqa: E731
    w1, w2 = rnd(E, 2 * I, H) / H ** 0.5, rnd(E, H, I) / I ** 0.5
    wc1, ws1 = qm.strata_moe_mxfp_quantize(w1.view(-1, H))
    wc2, ws2 = qm.strata_moe_mxfp_quantize(w2.view(-1, I))
    wc1, ws1, wc2, ws2 = (t.view(E, -1, t.shape[1]) for t in (wc1, ws1, wc2, ws2))
    h0 = rnd(T, H).to(torch.bfloat16)
    s = dict(h=h0.clone(), n1=qm.Norm(rnd(H), 1e-6), n2=qm.Norm(rnd(H), 1e-6), n3=qm.Norm(rnd(H), 1e-6, 1.0),
             x=torch.empty((T, H), device="cuda"), x2=torch.empty((T, H), device="cuda"), xc=u8(T, H // 2),
             xs=u8(T, H // 32), hid=torch.empty((T * K, I), device="cuda"), hc=u8(T * K, I // 2), hs=u8(T * K, I // 32),
             y=torch.empty((T * K, H), dtype=torch.bfloat16, device="cuda"),
             gate_up=qm.MxfpWeights(E, 2 * I, H, swiglu=True).pack(0, wc1, ws1),
             down=qm.MxfpWeights(E, H, I).pack(0, wc2, ws2))
    qm.strata_moe_norm_before(s["h"], s["n1"], s["x"])
    ids, s["p"] = qm.strata_moe_route(s["x"], rnd(H, E), None, K)
    s["offsets"], s["src"], slot = qm.strata_moe_group(ids, E)
    s["slot"] = slot.view(T, K)
    _layer(qm, s)
    n1 = _np(s["n1"].weight)
    want = ref.norm(_np(h0), n1, 0.0, 1e-6)
    _close(s["x"], want, np.abs(want))
    cuts, src = _np(s["offsets"]), _np(s["src"])
    c, b = ref.quantize(_np(s["x"]))
    xq = ref.values(c, b)[src]
    c, b = ref.quantize(_np(s["hid"]))
    assert np.array_equal(_np(s["hc"]), ref.pack(c)) and np.array_equal(_np(s["hs"]), b)
    hq = ref.values(c, b)
    for e in range(E):
        r = slice(cuts[e], cuts[e + 1])
        want, tol = ref.product(xq[r], ref.values(ref.unpack(_np(wc1[e])), _np(ws1[e])), True)
        assert np.all(np.abs(_np(s["hid"][r]) - want) <= tol + 2.0 ** -24 * (np.abs(want) + tol))
        want, tol = ref.product(hq[r], ref.values(ref.unpack(_np(wc2[e])), _np(ws2[e])), False)
        assert np.all(np.abs(_np(s["y"][r]) - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol))
    want, terms = _after_reference(dict(s, h=h0, gate=None), s["n2"].weight, 1.0, 0.5, 1e-6)
    _close(s["h"], want, terms)
    want = ref.norm(_np(s["h"]), _np(s["n3"].weight), 1.0, 1e-6)
    _close(s["x2"], want, np.abs(want))
    _check_codes(s["x2"], s["xc"], s["xs"])
    # captured; replayed on other streams' values with eager work between
    names = ("h", "x", "x2", "xc", "xs", "hid", "y")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _layer(qm, s)
    for i in range(3):
        start = rnd(T, H).to(torch.bfloat16)
        s["h"].copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        kept = {n: s[n].clone() for n in names}
        s["h"].copy_(start)
        _layer(qm, s)
        for n in names:
            assert torch.equal(kept[n], s[n]), n


@pytest.mark.gpu
def test_more_than_2_to_32_threads(qm):
    """4.2 million rows of 8192, a workgroup of 1024 each, a pattern of 1000 over and over."""
    T, H, part = (1 << 22) + 3, 8192, 1000
    torch.cuda.empty_cache()
    h = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")  # 69 GB
    few = torch.randn((part, H), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    for t in range(0, T, part):
        h[t:t + part] = few[:min(part, T - t)]
    codes = torch.empty((T, H // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
    norm = qm.Norm(torch.rand(H, generator=torch.Generator().manual_seed(2)).cuda())
    qm.strata_moe_norm_before(h, norm, codes=codes, scales=scales)
    c, s = torch.empty_like(codes[:part]), torch.empty_like(scales[:part])
    qm.strata_moe_norm_before(few, norm, codes=c, scales=s)
    for t in list(range(0, T, part * 61)) + [T // part * part]:
        k = min(part, T - t)
        assert torch.equal(codes[t:t + k], c[:k]) and torch.equal(scales[t:t + k], s[:k])
    del h, codes, scales
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ refusals
P = [(i + 1) << 24 for i in range(12)]


def _refused(qm, rc, code):
    assert rc == code and qm.strata_moe_last_error()


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), -1), (dict(T=(1 << 24) + 1), -1), (dict(H=0), -1), (dict(H=16385, h_stride=16385), -1),
    (dict(dtype=5), -2), (dict(h_stride=63), -1), (dict(h=None), -1), (dict(h=P[0] + 2), -1), (dict(x=P[1] + 2), -1),
    (dict(x=None, codes=None, scales=None), -1), (dict(codes=None), -1), (dict(scales=None), -1),
    (dict(codes=P[2] + 8), -1), (dict(H=40), -1), (dict(x=P[0]), -1), (dict(codes=P[0] + 16), -1),
    (dict(scales=P[1] + 9), -1), (dict(x=P[4]), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(offset=float("inf")), -1), (dict(weight=P[4] + 1), -1), (dict(norm=False), -1),
], ids=str)
def test_before_refuses(qm, change, code):
    a = dict(h=P[0], dtype=1, h_stride=64, T=8, H=64, x=P[1], codes=P[2], scales=P[3], weight=P[4], offset=0.0,
             eps=1e-6, norm=True)
    a.update(change)
    n = qm.NormStruct(a["weight"], a["offset"], a["eps"])
    _refused(qm, qm.library().strata_moe_norm_before(a["h"], a["dtype"], a["h_stride"], a["T"], a["H"],
                                                     ctypes.byref(n) if a["norm"] else None, a["x"], a["codes"],
                                                     a["scales"], None), code)


@pytest.mark.parametrize("change,code", [
    (dict(branch=False), -1), (dict(T=-1), -1), (dict(dtype=0), -2), (dict(y_dtype=0), -2), (dict(y_stride=63), -1),
    (dict(out_stride=63), -1), (dict(y_rows=-1), -1), (dict(y_rows=0), -1), (dict(slot=None), -1), (dict(p=None), -1),
    (dict(K=0), -1), (dict(K=17), -1), (dict(slot=None, p=None), -1), (dict(slot=None, p=None, K=0, y_rows=7), -1),
    (dict(rs=float("inf")), -1), (dict(bs=float("nan")), -1), (dict(gcol=2), -1), (dict(grow=-1), -1),
    (dict(out=None), -1), (dict(y=None), -1), (dict(out=P[5] + 2), -1), (dict(y=P[6] + 1), -1),
    (dict(slot=P[7] + 2), -1), (dict(p=P[8] + 2), -1), (dict(gate=P[9] + 2), -1), (dict(out=P[0] + 4), -1),
    (dict(out=P[0], out_stride=65), -1), (dict(out=P[6]), -1), (dict(out=P[7]), -1), (dict(x=P[0] + 64), -1),
    (dict(x=P[5]), -1), (dict(codes=P[9]), -1), (dict(next=False), -1), (dict(x=P[4]), -1), (dict(out=P[10]), -1),
    (dict(scales=P[8] + 5), -1),
], ids=str)
def test_after_refuses(qm, change, code):
    a = dict(h=P[0], dtype=1, h_stride=64, T=8, H=64, x=P[1], codes=P[2], scales=P[3], weight=P[4], out=P[5],
             out_stride=64, y=P[6], y_stride=64, y_rows=16, y_dtype=3, slot=P[7], p=P[8], K=2, gate=P[9], grow=64,
             gcol=1, next_weight=P[10], rs=1.0, bs=1.0, branch=True, next=True)
    a.update(change)
    n, u = qm.NormStruct(a["weight"], 0.0, 1e-6), qm.NormStruct(a["next_weight"], 0.0, 1e-6)
    b = qm.BranchStruct(a["y"], a["y_stride"], a["y_rows"], a["y_dtype"], a["K"], a["slot"], a["p"], ctypes.pointer(n),
                        a["gate"], a["grow"], a["gcol"], a["rs"], a["bs"])
    _refused(qm, qm.library().strata_moe_norm_after(
        a["h"], a["dtype"], a["h_stride"], a["T"], a["H"], ctypes.byref(b) if a["branch"] else None, a["out"],
        a["out_stride"], ctypes.byref(u) if a["next"] else None, a["x"], a["codes"], a["scales"], None), code)


def test_no_tokens_is_a_no_op(qm):
    lib = qm.library()
    n = qm.NormStruct(None, 0.0, 1e-6)
    assert lib.strata_moe_norm_before(None, 1, 64, 0, 64, ctypes.byref(n), P[0], None, None, None) == 0
    b = qm.BranchStruct(None, 64, 0, 1, 0, None, None, None, None, 0, 0, 1.0, 1.0)
    assert lib.strata_moe_norm_after(None, 1, 64, 0, 64, ctypes.byref(b), None, 64, None, None, None, None, None) == 0


@pytest.mark.parametrize("x,codes", [(None, None), (P[0], None), (None, P[1])])
def test_no_tokens_with_empty_arrays(qm, x, codes):
    """Arrays of no rows may be null: an allocation of no bytes is."""
    lib, n = qm.library(), qm.NormStruct(None, 0.0, 1e-6)
    scales = codes and P[2]
    assert lib.strata_moe_norm_before(None, 1, 64, 0, 64, ctypes.byref(n), x, codes, scales, None) == 0
    for K in (0, 1, 16):
        b = qm.BranchStruct(None, 64, 0, 1, K, None, None, None, None, 0, 0, 1.0, 1.0)
        for following in (None, ctypes.byref(n)):
            o = (x, codes, scales) if following else (None, None, None)
            assert lib.strata_moe_norm_after(None, 1, 64, 0, 64, ctypes.byref(b), None, 64, following, *o, None) == 0
    b = qm.BranchStruct(None, 64, 0, 1, 17, None, None, None, None, 0, 0, 1.0, 1.0)
    rc = lib.strata_moe_norm_after(None, 1, 64, 0, 64, ctypes.byref(b), None, 64, None, None, None, None, None)
    _refused(qm, rc, -1)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [0, 4])
def test_no_tokens_through_the_binding(qm, K):
    T, H, I, E = 0, 64, 96, 3
    f = lambda *a: torch.empty(a, device="cuda")  # noqa: E731
    u8 = lambda *a: torch.empty(a, dtype=torch.uint8, device="cuda")  # noqa: E731
    i32 = lambda *a: torch.empty(a, dtype=torch.int32, device="cuda")  # noqa: E731
    n = qm.Norm(torch.ones(H, device="cuda"))
    c, s = u8(T, H // 2), u8(T, H // 32)
    for x, codes, scales in ((f(T, H), None, None), (None, c, s), (f(T, H), c, s)):
        qm.strata_moe_norm_before(f(T, H), n, x, codes, scales)
        choice = dict(slot=i32(T, K), p=f(T, K)) if K else {}
        for gate in (None, f(H), f(T, 1), f(T, H)):
            for y in (f(T, H), f(5, H)) if K else (f(T, H),):
                qm.strata_moe_norm_after(f(T, H), y, f(T, H), norm=n, gate=gate, next_norm=n, x=x, codes=codes,
                                         scales=scales, **choice)
    codes, scales = qm.strata_moe_mxfp_quantize(f(T, H))
    assert qm.strata_moe_mxfp_dequantize(codes, scales, f(T, H)).shape == (T, H)
    w = qm.MxfpWeights(E, I, H).pack(0, u8(0, I, H // 2), u8(0, I, H // 32))
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    for x_rows in (0, 5):
        out = qm.strata_moe_mxfp_product(u8(x_rows, H // 2), u8(x_rows, H // 32), w, f(0, I), offsets=off, src=i32(0))
        assert out.shape == (0, I)
    torch.cuda.synchronize()


def test_no_choices_are_not_no_combine(qm):
    """slot and p of [T][0]: their memory is a null pointer, which to the library says that there are none."""
    h = torch.zeros((4, 64))
    none = dict(slot=torch.zeros((4, 0), dtype=torch.int32), p=torch.zeros((4, 0)))
    for rows in (4, 9):
        with pytest.raises(ValueError):
            qm.strata_moe_norm_after(h, torch.zeros((rows, 64)), h.clone(), **none)


def test_the_binding_checks_its_tensors(qm):
    h, x = torch.zeros((4, 64)), torch.zeros((4, 64))
    n = qm.Norm(None)
    with pytest.raises(TypeError):
        qm.strata_moe_norm_before(h, n, x)                  # not on the GPU
    with pytest.raises(TypeError):
        qm.strata_moe_norm_before(h, None, x)
    with pytest.raises(TypeError):
        qm.strata_moe_norm_before(h.double(), n, x)
    with pytest.raises(ValueError):
        qm.strata_moe_norm_before(h, n, x[:3])
    with pytest.raises(ValueError):
        qm.strata_moe_norm_before(h, qm.Norm(torch.zeros(63)), x)
    with pytest.raises(TypeError):
        qm.Norm(torch.zeros(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        qm.strata_moe_norm_before(h, n, x, codes=torch.zeros((4, 32), dtype=torch.uint8))
    with pytest.raises(ValueError):
        qm.strata_moe_norm_after(h, h[:3], x)
    with pytest.raises(TypeError):
        qm.strata_moe_norm_after(h, h, x.half())
    with pytest.raises(ValueError):
        qm.strata_moe_norm_after(h, h, x, slot=torch.zeros((4, 1), dtype=torch.int32))
    for gate in (torch.zeros(63), torch.zeros((4, 2)), torch.zeros((3, 1)), torch.zeros((64, 4)).t()):
        with pytest.raises(ValueError):
            qm.strata_moe_norm_after(h, h, x, gate=gate)
