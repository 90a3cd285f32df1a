"""Microscaled 4-bit floating point (strata_moe_mxfp_*) against its definition in
64 bits: rounding and packing bit for bit, products within the tolerance that
mxfp_reference.product derives, plus half a step of the output's type."""
import ctypes

import mxfp_reference as ref
import numpy as np
import pytest
import torch

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
IDS = ["fp32", "fp16", "bf16"]


@pytest.fixture(scope="module")
def qm():
    import quantized_routed_expert_logits_amd as qm
    return qm


def _np(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


# ------------------------------------------------------------------ rounding
def _check_quantize(qm, x):
    codes, scales = qm.strata_moe_mxfp_quantize(x)
    want, byte = ref.quantize(_np(x))
    assert np.array_equal(_np(scales), byte)
    assert np.array_equal(_np(codes), ref.pack(want))
    return codes, scales


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,cols,pad",
                         [(1, 32, 0), (1, 2560, 0), (3, 64, 1), (7, 96, 8), (33, 1056, 3), (130, 544, 0),
                                           (1025, 32, 5), (2, 65536, 0), (600, 2560, 0)])
def test_quantize(qm, rows, cols, pad, dtype):
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn((rows, cols + pad), generator=g) * torch.exp2(torch.randint(-9, 6, (rows, 1), generator=g).float())
    x = x.to(dtype).cuda()[:, :cols]
    codes, scales = _check_quantize(qm, x)
    for dt in DTYPES:  # read back, into padded rows
        buf = torch.full((rows, cols + 3), 7.0, dtype=dt, device="cuda")
        out = qm.strata_moe_mxfp_dequantize(codes, scales, buf[:, :cols])
        v = ref.values(ref.unpack(_np(codes)), _np(scales))
        assert torch.equal(out.cpu(), torch.from_numpy(v).to(dt))
        assert torch.all(buf[:, cols:] == 7.0)


@pytest.mark.gpu
def test_quantize_every_border(qm):
    """Values on, just above and just below every border between two codes, in
    blocks whose largest value spans all exponents."""
    marks = np.array([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0, 7.9999995],
                     np.float32)
    near = np.concatenate([marks, np.nextafter(marks, np.float32(9)), np.nextafter(marks, np.float32(-9))])
    near = np.concatenate([near, -near])
    rows = []
    for e in list(range(-149, -120)) + [-60, -1, 0, 1, 77, 123, 125]:
        with np.errstate(over="ignore", under="ignore"):
            v = (near.astype(np.float64) * 2.0 ** e).astype(np.float32)
            top = np.float32(7.0 * 2.0 ** e)
        v = v[np.abs(v) <= max(top, np.float32(2.0 ** -149))]
        for i in range(0, len(v), 31):
            block = np.zeros(32, np.float32)
            block[:len(v[i:i + 31])] = v[i:i + 31]
            block[31] = top
            rows.append(block)
    x = torch.from_numpy(np.stack(rows)).cuda()
    assert torch.isfinite(x).all()
    _check_quantize(qm, x)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_quantize_infinities_and_nan_stay_in_their_block(qm, dtype):
    x = torch.randn((4, 128), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    x[0, 5], x[1, 40], x[2, 127] = float("inf"), float("nan"), -float("inf")
    x[3] = 0.0
    codes, scales = _check_quantize(qm, x)
    v = qm.strata_moe_mxfp_dequantize(codes, scales, torch.empty_like(x))
    nan = torch.isnan(v)
    assert nan.sum() == 96 and nan[0, :32].all() and nan[1, 32:64].all() and nan[2, 96:].all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_every_code_at_every_scale_is_read_back(qm, dtype):
    """Rounded to the type: infinite past it, subnormal and zero below, NaN at byte 255."""
    codes = np.broadcast_to(np.arange(32, dtype=np.uint8) % 16, (256, 32))
    byte = np.arange(256, dtype=np.uint8)[:, None]
    out = qm.strata_moe_mxfp_dequantize(torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(byte).cuda(),
                                        torch.empty((256, 32), dtype=dtype).cuda())
    v = ref.values(codes, byte)
    want = torch.from_numpy(v).to(dtype)
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(want))
    assert torch.equal(out[:255].cpu(), want[:255])
    if dtype != torch.float16:  # exact, but for magnitudes 4 and 6 at byte 253 and 2 to 6 at 254
        past = (byte == 253) & (codes % 8 >= 6) | (byte == 254) & (codes % 8 >= 4)
        exact = want.double().numpy() == v
        assert exact[:255][~past[:255]].all() and torch.isinf(want[torch.from_numpy(past)]).all()


# ------------------------------------------------------------------- product
def _operands(rows, cols, n, E, seed, spread=6):
    g = torch.Generator().manual_seed(seed)
    xc = torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.uint8)
    xs = torch.randint(127 - spread, 127 + spread, (rows, cols // 32), generator=g, dtype=torch.uint8)
    wc = torch.randint(0, 256, (E, n, cols // 2), generator=g, dtype=torch.uint8)
    ws = torch.randint(120 - spread, 120 + spread, (E, n, cols // 32), generator=g, dtype=torch.uint8)
    return xc.cuda(), xs.cuda(), wc.cuda(), ws.cuda()


def _offsets(E, rows, seed, how="random"):
    g = np.random.default_rng(seed)
    if how == "one":  # all rows to one expert in the middle
        n = np.zeros(E, np.int64)
        n[E // 2] = rows
    elif how == "hot":  # half of the rows to the last expert
        n = np.bincount(np.where(g.random(rows) < 0.5, E - 1, g.integers(0, E, rows)), minlength=E)
    else:
        n = np.bincount(g.integers(0, E, rows), minlength=E)
    return torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()


def _check_product(qm, xc, xs, wc, ws, out, swiglu=False, offsets=None, src=None, weights=None, only=None):
    """out (given, holds what an untouched element keeps) after the call, against the definition."""
    before = _np(out)
    E, n, _ = wc.shape
    if weights is None:
        weights = qm.MxfpWeights(E, n, xc.shape[1] * 2, swiglu=swiglu).pack(0, wc, ws)
    qm.strata_moe_mxfp_product(xc, xs, weights, out, offsets=offsets, src=src)
    got, dt = _np(out), torch.finfo(out.dtype)
    x = ref.values(ref.unpack(_np(xc)), _np(xs))
    rows = np.arange(out.shape[0]) if src is None else _np(src)
    cuts = [0, out.shape[0]] if offsets is None else _np(offsets)
    want, tol, written = before.copy(), np.zeros_like(got), np.zeros(out.shape[0], bool)
    for e in range(E) if only is None else only:
        r = np.arange(cuts[e], cuts[e + 1])
        if len(r) == 0:
            continue
        xe = np.where(((rows[r] >= 0) & (rows[r] < len(x)))[:, None], x[np.clip(rows[r], 0, len(x) - 1)], 0.0)
        w = ref.values(ref.unpack(_np(wc[e])), _np(ws[e]))
        want[r], t = ref.product(xe, w, swiglu)
        tol[r] = t + ref.rounding(dt.eps, dt.smallest_normal * dt.eps, np.abs(want[r]) + t)
        written[r] = True
    if only is None:
        assert np.array_equal(got[~written], before[~written]), "a row of no expert changed"
    err = np.abs(got - want)[written]
    # rounding to nearest gives infinity from the largest value and half a step on: half a step is
    # eps / 2 of that value's power of two, (2 - eps) of which is the largest value
    border = dt.max * (1.0 + dt.eps / 2 / (2.0 - dt.eps))
    over = np.isinf(got) & (np.abs(want) + tol >= border) & (np.sign(got) == np.sign(want))
    bad = ~((err <= tol[written]) | over[written])
    worst = np.nanmax(np.where(over[written], 0.0, err) / np.maximum(tol[written], 1e-300))
    assert not bad.any(), f"{bad.sum()} outputs off, worst {worst:.2f} of the tolerance"


DENSE = [  # rows, cols, n
    (1, 32, 1), (1, 2560, 2560), (2, 64, 15), (5, 96, 17), (16, 128, 64), (17, 544, 333), (31, 640, 65),
    (64, 1024, 100), (65, 512, 256), (128, 160, 257), (129, 1056, 128), (200, 2560, 320), (300, 4096, 96),
    (3, 65536, 20), (2, 32, 65536), (1000, 96, 70), (2049, 512, 130),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("size", DENSE, ids=lambda s: "-".join(map(str, s)))
def test_product_of_one_matrix(qm, size, dtype):
    rows, cols, n = size
    xc, xs, wc, ws = _operands(rows, cols, n, 1, seed=rows + n)
    buf = torch.full((rows, n + 3), 7.0, dtype=dtype, device="cuda")
    _check_product(qm, xc, xs, wc, ws, buf[:, :n])
    assert torch.all(buf[:, n:] == 7.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("size",
                         [(1, 32, 2), (1, 2560, 2048), (9, 96, 30), (17, 544, 34), (130, 640, 512), (257, 512, 666)],
                         ids=lambda s: "-".join(map(str, s)))
def test_swiglu_of_one_matrix(qm, size, dtype):
    rows, cols, n = size
    # large scales: gates on both sides of where the exponential overflows
    xc, xs, wc, ws = _operands(rows, cols, n, 1, seed=rows + n, spread=3)
    buf = torch.full((rows, n // 2 + 1), 7.0, dtype=dtype, device="cuda")
    _check_product(qm, xc, xs, wc, ws, buf[:, :n // 2], swiglu=True)
    assert torch.all(buf[:, n // 2:] == 7.0)


GROUPED = [  # rows, x rows (0: no src), cols, n, E, how, swiglu
    (1, 1, 96, 32, 512, "random", True), (10, 1, 2560, 128, 512, "random", True),
    (10, 0, 1024, 80, 512, "random", False), (64, 20, 160, 33, 7, "random", False),
    (406, 203, 544, 333, 6, "random", False), (300, 30, 640, 64, 1024, "random", True),
    (320, 32, 256, 96, 512, "random", False), (1000, 100, 128, 48, 40, "hot", True), (777, 0, 96, 20, 5, "one", False),
    (2000, 500, 512, 260, 16, "random", True), (1500, 0, 672, 300, 9, "hot", False),
    (4000, 400, 96, 16, 1024, "hot", False), (520, 52, 64, 40, 3, "one", True), (33, 33, 2560, 64, 2, "random", False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("size", GROUPED, ids=lambda s: "-".join(map(str, s)))
def test_product_by_expert(qm, size):
    rows, x_rows, cols, n, E, how, swiglu = size
    xc, xs, wc, ws = _operands(x_rows or rows, cols, n, E, seed=rows)
    src = torch.randint(0, x_rows, (rows,), generator=torch.Generator().manual_seed(3)).int().cuda() if x_rows else None
    for dtype in DTYPES:
        out = torch.full((rows, n // 2 if swiglu else n), 7.0, dtype=dtype, device="cuda")
        _check_product(qm, xc, xs, wc, ws, out, swiglu=swiglu, offsets=_offsets(E, rows, rows, how), src=src)


# On both sides of each border between the product's kernels (by rows and runs of
# 64 weight rows, then by 16-row tiles, runs and steps) and between the item sizes
# of the kernel of many rows.
BORDERS = [  # rows, cols, n, E (0: no offsets)
    (512, 64, 60, 7), (513, 64, 60, 7), (512, 96, 1024, 0), (513, 96, 1024, 0),
    (592, 512, 2560, 0), (593, 512, 2560, 0), (6000, 32, 1024, 0), (6001, 32, 1024, 0),
    (2048, 512, 1024, 0), (2049, 512, 1024, 0), (4096, 512, 1000, 0), (4097, 512, 1000, 0),
    (1984, 1024, 700, 8), (2048, 1024, 700, 3), (9000, 512, 700, 8),
]


@pytest.mark.gpu
@pytest.mark.parametrize("size", BORDERS, ids=lambda s: "-".join(map(str, s)))
def test_borders_between_kernels(qm, size):
    rows, cols, n, E = size
    xc, xs, wc, ws = _operands(rows, cols, n, E or 1, seed=rows + n)
    out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
    _check_product(qm, xc, xs, wc, ws, out, offsets=_offsets(E, rows, rows) if E else None)


MANY = [  # rows, x rows (0: no src), cols, n, E, how, swiglu: all taken by the kernel of many rows
    (3600, 0, 544, 334, 0, "", True), (1500, 0, 640, 2047, 0, "", False), (1300, 0, 4128, 515, 0, "", False),
    (4000, 400, 512, 256, 1024, "random", True), (4000, 0, 672, 250, 1024, "hot", False),
    (4000, 203, 544, 334, 6, "random", True), (2600, 7, 1056, 400, 5, "one", False),
    (5000, 4, 32, 2048, 4, "random", False), (7000, 11, 96, 1024, 3, "hot", True),
    (1800, 257, 2560, 96, 64, "random", True), (3000, 3001, 480, 512, 2, "random", False),
    (1000, 0, 1536, 1100, 1, "one", True), (20000, 0, 512, 640, 3, "random", False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("size", MANY, ids=lambda s: "-".join(map(str, s)))
def test_product_of_many_rows(qm, size, dtype):
    """With rows that src names twice or not at all, or that lie outside x, with
    output rows that do and do not take 16-byte stores, and with scales that begin
    at an odd byte."""
    rows, x_rows, cols, n, E, how, swiglu = size
    xc, xs, wc, ws = _operands(x_rows or rows, cols, n, E or 1, seed=rows)
    odd = torch.full((xs.numel() + 1,), 255, dtype=torch.uint8, device="cuda")[1:].view(xs.shape)
    odd.copy_(xs)
    src = None
    if x_rows:
        g = torch.Generator().manual_seed(3)
        src = torch.randint(0, x_rows, (rows,), generator=g).int()
        src[torch.randint(0, rows, (9,), generator=g)] = -1
        src[torch.randint(0, rows, (9,), generator=g)] = x_rows
        src = src.cuda()
    n_out = n // 2 if swiglu else n
    offsets = _offsets(E, rows, rows, how) if E else None
    weights = qm.MxfpWeights(max(E, 1), n, cols, swiglu=swiglu).pack(0, wc, ws)
    outs = []
    for pad in (3, 16 + -n_out % 16):
        buf = torch.full((rows, n_out + pad), 7.0, dtype=dtype, device="cuda")
        _check_product(qm, xc, odd, wc, ws, buf[:, :n_out], swiglu=swiglu, offsets=offsets, src=src, weights=weights)
        assert torch.all(buf[:, n_out:] == 7.0)
        outs.append(buf[:, :n_out])
    assert torch.equal(outs[0], outs[1])


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [512, 544])
def test_runs_of_rows_outside_x(qm, cols):
    """Several items in turn per workgroup, of which every other one has rows that
    count as zeros, and the ones between have none."""
    rows, n = 24000, 1024
    xc, xs, wc, ws = _operands(300, cols, n, 1, seed=12)
    r = torch.arange(rows)
    src = torch.where(r // 96 % 2 == 1, (r % 5 - 1) * 1000, r % 300).int()  # outside x but for 0
    out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
    _check_product(qm, xc, xs, wc, ws, out, src=src.cuda())


@pytest.mark.gpu
def test_two_products_at_once(qm):
    """The same weights and rows on two streams, and one of few rows beside them."""
    xc, xs, wc, ws = _operands(2000, 640, 400, 6, seed=13)
    w = qm.MxfpWeights(6, 400, 640).pack(0, wc, ws)
    off = _offsets(6, 2000, 4)
    want = qm.strata_moe_mxfp_product(xc, xs, w, torch.empty((2000, 400), device="cuda"), offsets=off)
    small = torch.tensor([0, 2, 2, 3, 3, 3, 4], dtype=torch.int32, device="cuda")
    few = qm.strata_moe_mxfp_product(xc[:4], xs[:4], w, torch.empty((4, 400), device="cuda"), offsets=small)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.zeros((2000, 400), device="cuda") for _ in range(2)] + [torch.zeros((4, 400), device="cuda")]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, o in zip(streams, outs):
            k = o.shape[0]
            qm.strata_moe_mxfp_product(xc[:k], xs[:k], w, o, offsets=off if k > 4 else small, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want) and torch.equal(outs[2], few)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [40, 900])
def test_rows_of_no_expert_are_left(qm, rows):
    xc, xs, wc, ws = _operands(rows, 96, 40, 4, seed=1)
    off = torch.tensor([7, 7, 19, 19, rows - 5], dtype=torch.int32, device="cuda")
    _check_product(qm, xc, xs, wc, ws, torch.full((rows, 40), 7.0, device="cuda"), offsets=off)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [30, 700])
def test_src_outside_x_counts_as_zeros(qm, rows):
    xc, xs, wc, ws = _operands(9, 160, 50, 3, seed=2)
    src = torch.randint(-3, 12, (rows,), generator=torch.Generator().manual_seed(0)).int()
    src[0], src[1], src[2] = -2 ** 31, 2 ** 31 - 1, 9
    out = torch.full((rows, 50), 7.0, device="cuda")
    _check_product(qm, xc, xs, wc, ws, out, offsets=_offsets(3, rows, 5), src=src.cuda())


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [20, 400])
def test_offsets_of_any_value_stay_in_the_arrays(qm, rows):
    """Offsets that fall, are negative or lie past the rows: nothing outside out
    is written, and an expert whose range is in order gets its rows."""
    xc, xs, wc, ws = _operands(rows, 64, 24, 5, seed=3)
    w = qm.MxfpWeights(5, 24, 64).pack(0, wc, ws)
    buf = torch.full((rows + 64, 24), 7.0, device="cuda")
    off = torch.tensor([-2 ** 31, 4, 2, 2 ** 31 - 1, -7, 3], dtype=torch.int32, device="cuda")
    qm.strata_moe_mxfp_product(xc, xs, w, buf[:rows], offsets=off)
    assert torch.all(buf[rows:] == 7.0)
    x = ref.values(ref.unpack(_np(xc)), _np(xs))
    want, tol = ref.product(x[5:], ref.values(ref.unpack(_np(wc[2])), _np(ws[2])),
                            False)  # rows 5.. are expert 2's alone
    assert np.all(np.abs(_np(buf[5:rows]) - want) <= tol + 2.0 ** -24 * np.abs(want))


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [12, 300])
def test_nan_stays_in_its_row_and_output(qm, rows):
    xc, xs, wc, ws = _operands(rows, 256, 48, 1, seed=4)
    xs[3, 7], ws[0, 20, 1] = 255, 255
    out = torch.empty((rows, 48), device="cuda")
    qm.strata_moe_mxfp_product(xc, xs, qm.MxfpWeights(1, 48, 256).pack(0, wc, ws), out)
    want = torch.zeros((rows, 48), dtype=torch.bool, device="cuda")
    want[3], want[:, 20] = True, True
    assert torch.equal(torch.isnan(out), want)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [5, 140])
def test_a_row_s_result_does_not_depend_on_its_neighbours(qm, rows):
    """The padding of a step and of a tile reads nothing: the same row beside NaN
    rows and before the end of the array."""
    xc, xs, wc, ws = _operands(rows, 544, 70, 1, seed=5)
    w = qm.MxfpWeights(1, 70, 544).pack(0, wc, ws)
    out = qm.strata_moe_mxfp_product(xc, xs, w, torch.empty((rows, 70), device="cuda"))
    xs2 = xs.clone()
    xs2[1::2] = 255
    out2 = qm.strata_moe_mxfp_product(xc, xs2, w, torch.empty((rows, 70), device="cuda"))
    assert torch.equal(out[0::2], out2[0::2]) and torch.isnan(out2[1::2]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows", [64, 960, 2500])  # a workgroup per row and run, the list, the kernel of many rows
def test_swiglu_over_the_whole_range(qm, rows, dtype):
    """Gates to both ends of fp32 and past them, with ups of every size: the gate and
    the up of an output are sums of two products that are exact in fp32."""
    two = (0.0, 0)  # (magnitude, exponent) of a product
    gates = [((1.0, 127), (1.5, 125)), ((1.0, 127), (1.5, 126)), ((1.5, 127), two), ((1.5, 127), (1.5, 125)),
             ((6.0, 127), two), ((1.0, 6), (1.5, 4)), ((1.0, 0), two), (two, two), ((1.5, 100), two)]
    ups = [((1.0, -33), two), ((1.5, -100), two), ((1.0, 0), two), ((1.5, 14), (1.0, 3)), ((1.0, 100), two),
           ((6.0, 127), two), (two, two)]
    pairs = [(g, u) for g in gates for u in ups]
    n = 320
    pairs = [pairs[j % len(pairs)] for j in range(n)]
    code = {0.0: 0, 1.0: 2, 1.5: 3, 6.0: 7}
    wc, ws = torch.zeros((1, 2 * n, 64), dtype=torch.uint8), torch.full((1, 2 * n, 4), 127, dtype=torch.uint8)
    sums = np.zeros(2 * n)
    for j, pair in enumerate(pairs):
        for half in range(2):
            for i, (m, e) in enumerate(pair[half]):  # x is 2^63 in the gates' blocks, 1 in the ups'
                b, row = 2 * half + i, half * n + j
                byte = e + 127 - (0 if half or m == 0.0 else 63)
                assert 0 <= byte <= 254
                wc[0, row, 16 * b], ws[0, row, b] = code[m], byte
                sums[row] += m * 2.0 ** e
    xc, xs = torch.zeros((rows, 64), dtype=torch.uint8), torch.full((rows, 4), 127, dtype=torch.uint8)
    sign = np.where(np.arange(rows) % 3 == 1, -1.0, 1.0)
    xc[:, ::16] = torch.from_numpy(np.where(sign < 0, 10, 2).astype(np.uint8))[:, None]
    xs[:, :2] = 63 + 127
    weights = qm.MxfpWeights(1, 2 * n, 128, swiglu=True).pack(0, wc.cuda(), ws.cuda())
    out = _np(qm.strata_moe_mxfp_product(xc.cuda(), xs.cuda(), weights, torch.empty((rows, n), dtype=dtype).cuda()))
    with np.errstate(all="ignore"):
        y = (sign[:, None] * sums).astype(np.float32).astype(np.float64)  # infinite from 2^128 on
        g, u = y[:, :n], y[:, n:]
        want = g / (1.0 + np.exp(-g)) * u
        # the output's rounding, and the arithmetic as ref.product has it: 12 roundings, 0 below -87
        fi = torch.finfo(dtype)
        tol = ref.rounding(fi.eps, fi.smallest_normal * fi.eps, want) + 12 * 2.0 ** -23 * np.abs(want)
        tol = np.where(g < -87, tol + 2.0 ** -118 * np.abs(u), tol)
        border = fi.max * (1.0 + fi.eps / 2 / (2.0 - fi.eps))  # from here on the nearest is infinity
        over = np.isinf(out) & (np.abs(want) + tol >= border) & (np.sign(out) == np.sign(want))
        ok = (np.abs(out - want) <= tol) | over | (np.isnan(out) & np.isnan(want))
    ok |= (g < -87) & (g > -100) & np.isinf(u)  # 0 times infinity there: 0 is what the gate may be
    assert ok.all(), [(g[i], u[i], out[i], want[i]) for i in map(tuple, np.argwhere(~ok)[:5])]


@pytest.mark.gpu
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("rows,n", [(30, 50), (700, 50), (4000, 400)])  # one in each of the three kernels
def test_src_outside_x_gives_zeros_whatever_the_weights(qm, rows, n, swiglu):
    """Weights that hold NaN blocks: a row with a source is NaN at their outputs, a row without one 0 everywhere."""
    xc, xs, wc, ws = _operands(9, 160, n, 3, seed=20)
    for e in range(3):
        ws[e, e::7, e] = 255
    src = torch.randint(-3, 12, (rows,), generator=torch.Generator().manual_seed(21)).int()
    src[0], src[1] = -2 ** 31, 2 ** 31 - 1
    off = _offsets(3, rows, 22)
    n_out = n // 2 if swiglu else n
    out = torch.full((rows, n_out), 7.0, device="cuda")
    qm.strata_moe_mxfp_product(xc, xs, qm.MxfpWeights(3, n, 160, swiglu=swiglu).pack(0, wc, ws), out, offsets=off,
                               src=src.cuda())
    nan = (ws == 255).any(-1).cpu()
    nan = nan[:, :n_out] | nan[:, -n_out:]
    expert = torch.bucketize(torch.arange(rows, dtype=torch.int32), off.cpu()[1:], right=True)
    outside = (src < 0) | (src >= 9)
    out = out.cpu()
    assert torch.all(out[outside] == 0)
    assert torch.equal(torch.isnan(out[~outside]), nan[expert[~outside]])


# The next three with sizes for the list and for the kernel of many rows: rows, cols, n.
@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,n", [(9000, 256, 48), (3000, 256, 600), (3000, 544, 600), (10000, 32, 1000)])
def test_nan_stays_in_its_row_and_output_of_many(qm, rows, cols, n):
    xc, xs, wc, ws = _operands(rows, cols, n, 1, seed=23)
    xs[3, -1], xs[rows - 1, 0], ws[0, 20, 0], ws[0, n - 1, -1] = 255, 255, 255, 255
    out = torch.empty((rows, n), device="cuda")
    qm.strata_moe_mxfp_product(xc, xs, qm.MxfpWeights(1, n, cols).pack(0, wc, ws), out)
    want = torch.zeros((rows, n), dtype=torch.bool, device="cuda")
    want[3], want[rows - 1], want[:, 20], want[:, n - 1] = True, True, True, True
    assert torch.equal(torch.isnan(out), want)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,n", [(9000, 544, 70), (3000, 544, 600), (10000, 32, 1000), (5000, 96, 1000),
                                         (3000, 608, 600), (3000, 672, 600), (3000, 992, 600), (3001, 1056, 600)])
def test_many_rows_do_not_depend_on_their_neighbours(qm, rows, cols, n):
    """Every other row NaN, where a group of 512 ends after 1, 2, 3, 5 and 15 blocks: behind a row's
    last scale the next row's are read, and left out."""
    xc, xs, wc, ws = _operands(rows, cols, n, 1, seed=24)
    w = qm.MxfpWeights(1, n, cols).pack(0, wc, ws)
    alone = torch.empty((rows, n), device="cuda")
    _check_product(qm, xc, xs, wc, ws, alone, weights=w)
    for odd in (1, 0):
        xs2 = xs.clone()
        xs2[odd::2] = 255
        out = qm.strata_moe_mxfp_product(xc, xs2, w, torch.empty((rows, n), device="cuda"))
        assert torch.equal(out[1 - odd::2], alone[1 - odd::2]) and torch.isnan(out[odd::2]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,n", [(900, 64, 24), (8000, 64, 700), (8000, 544, 700)])
def test_offsets_of_any_value_with_many_rows(qm, rows, cols, n):
    """Offsets that fall, are negative or lie past the rows, and offsets with gaps, also with NaN
    rows and weights beside the rows that have an expert."""
    xc, xs, wc, ws = _operands(rows, cols, n, 5, seed=25)
    w = qm.MxfpWeights(5, n, cols).pack(0, wc, ws)
    buf = torch.full((rows + 64, n), 7.0, device="cuda")
    off = torch.tensor([-2 ** 31, 4, 2, 2 ** 31 - 1, -7, 3], dtype=torch.int32, device="cuda")
    qm.strata_moe_mxfp_product(xc, xs, w, buf[:rows], offsets=off)
    assert torch.all(buf[rows:] == 7.0)
    x = ref.values(ref.unpack(_np(xc)), _np(xs))[4:]  # rows 4.. are expert 2's alone
    want, tol = ref.product(x, ref.values(ref.unpack(_np(wc[2])), _np(ws[2])), False)
    assert np.all(np.abs(_np(buf[4:rows]) - want) <= tol + 2.0 ** -24 * (np.abs(want) + tol))
    off = torch.tensor([7, 7, 19, 19, rows // 2, rows - 5], dtype=torch.int32, device="cuda")
    xs[:7], xs[rows - 5:], ws[0], ws[2] = 255, 255, 255, 255
    _check_product(qm, xc, xs, wc, ws, torch.full((rows, n), 7.0, device="cuda"), offsets=off)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n_e", [(3, 1), (50, 8), (3000, 8)])
def test_repeated_calls_give_the_same_bits(qm, rows, n_e):
    xc, xs, wc, ws = _operands(rows, 640, 200, n_e, seed=6)
    w = qm.MxfpWeights(n_e, 200, 640, swiglu=True).pack(0, wc, ws)
    off = None if n_e == 1 else _offsets(n_e, rows, 1)
    outs = [qm.strata_moe_mxfp_product(xc, xs, w, torch.empty((rows, 100), device="cuda"),
                                       offsets=off) for _ in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [6, 600])
def test_graph_and_streams(qm, rows):
    """Captured with the rounding before it and replayed with new inputs, beside
    the same call on another stream."""
    g = torch.Generator().manual_seed(7)
    E, cols, n = 5, 672, 96
    _, _, wc, ws = _operands(1, cols, n, E, seed=8)
    w = qm.MxfpWeights(E, n, cols).pack(0, wc, ws)
    off = _offsets(E, rows, 2)
    x = torch.randn((rows, cols), generator=g).cuda()
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device="cuda")
    out = torch.empty((rows, n), device="cuda")

    def call(stream=None):
        qm.strata_moe_mxfp_quantize(x, codes, scales, stream=stream)
        qm.strata_moe_mxfp_product(codes, scales, w, out, offsets=off, stream=stream)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    side = torch.cuda.Stream()
    for i in range(4):
        x.copy_(torch.randn((rows, cols), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        c2, s2 = qm.strata_moe_mxfp_quantize(x)
        eager = qm.strata_moe_mxfp_product(c2, s2, w, torch.empty_like(out), offsets=off)
        side.wait_stream(torch.cuda.current_stream())
        other = torch.empty_like(out)
        c3, s3 = qm.strata_moe_mxfp_quantize(x, stream=side)
        qm.strata_moe_mxfp_product(c3, s3, w, other, offsets=off, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(out, other)


@pytest.mark.gpu
def test_weights_and_outputs_past_32_bits(qm):
    E, n, cols = 900, 4096, 2560  # 5 GB of packed weights
    g = torch.Generator(device="cuda").manual_seed(9)
    w = qm.MxfpWeights(E, n, cols)
    wc = torch.randint(0, 256, (E, n, cols // 2), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.randint(114, 126, (E, n, cols // 32), generator=g, device="cuda", dtype=torch.uint8)
    w.pack(0, wc, ws)
    assert w.packed.numel() > 1 << 32
    xc, xs, _, _ = _operands(6, cols, 1, 1, seed=10)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:], off[500:], off[900:] = 1, 3, 6  # experts 0, 499 and 899
    _check_product(qm, xc, xs, wc, ws, torch.empty((6, n), device="cuda"), offsets=off.cuda(), weights=w,
                   only=[0, 499, 899])
    del wc, ws, w
    rows = 1100000  # 4.5e9 outputs
    xc, xs, wc, ws = _operands(64, 32, n, 1, seed=11)
    src = (torch.arange(rows, device="cuda") % 64).int()
    out = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
    qm.strata_moe_mxfp_product(xc, xs, qm.MxfpWeights(1, n, 32).pack(0, wc, ws), out, src=src)
    first = torch.empty((64, n), dtype=torch.bfloat16, device="cuda")
    _check_product(qm, xc, xs, wc, ws, first)
    for r0 in (0, 524288, 1048512, rows - rows % 64 - 64):
        assert torch.equal(out[r0:r0 + 64], first)
    assert torch.equal(out[rows - rows % 64:], first[:rows % 64])


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [9, 6200])
def test_rows_of_x_past_32_bits(qm, rows):
    """Rows all over an x whose codes fill 4 GB, against the same rows by themselves."""
    x_rows, cols, n = (1 << 24) - 1, 512, 256
    g = torch.Generator(device="cuda").manual_seed(14)
    xc = torch.randint(0, 256, (x_rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8)
    xs = torch.randint(120, 130, (x_rows, cols // 32), generator=g, device="cuda", dtype=torch.uint8)
    _, _, wc, ws = _operands(1, cols, n, 1, seed=15)
    w = qm.MxfpWeights(1, n, cols).pack(0, wc, ws)
    src = torch.randint(0, x_rows, (rows,), generator=g, device="cuda").int()
    src[:4] = torch.tensor([x_rows - 1, 0, x_rows - 2, 1 << 23], dtype=torch.int32)
    out = qm.strata_moe_mxfp_product(xc, xs, w, torch.empty((rows, n), device="cuda"), src=src)
    alone = torch.empty((rows, n), device="cuda")
    _check_product(qm, xc[src.long()], xs[src.long()], wc, ws, alone, weights=w)
    assert torch.equal(out, alone)


@pytest.mark.gpu
def test_rounding_past_32_bits(qm):
    rows, cols = (1 << 24) - 1, 1000 // 32 * 32  # 1.7e10 values, 33 GB
    part = _float_part(4099, cols)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    for r in range(0, rows, 4099):
        x[r:r + 4099] = part[:min(4099, rows - r)]
    codes, scales = qm.strata_moe_mxfp_quantize(x)
    want = _check_quantize(qm, part)
    back = qm.strata_moe_mxfp_dequantize(codes, scales, x)
    values = qm.strata_moe_mxfp_dequantize(*want, torch.empty_like(part))
    for r in list(range(0, rows, 4099 * 97)) + [rows // 4099 * 4099]:
        k = min(4099, rows - r)
        assert torch.equal(codes[r:r + k], want[0][:k]) and torch.equal(scales[r:r + k], want[1][:k])
        assert torch.equal(back[r:r + k], values[:k])


def _float_part(rows, cols):
    g = torch.Generator().manual_seed(rows)
    return torch.randn((rows, cols), generator=g).to(torch.bfloat16).cuda()


# ------------------------------------------------------------------ refusals
PTR = 1 << 20


def _refused(qm, rc, code):
    assert rc == code and qm.strata_moe_last_error()


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), -1), (dict(rows=(1 << 24) + 1), -1), (dict(cols=0), -1), (dict(cols=48), -1),
    (dict(cols=65568), -1), (dict(dtype=0), -2), (dict(dtype=4), -2), (dict(x_stride=63), -1),
    (dict(x_stride=(1 << 32) + 1), -1), (dict(x=None), -1), (dict(codes=None), -1), (dict(scales=None), -1),
    (dict(x=PTR + 2), -1), (dict(codes=(2 << 20) + 8), -1), (dict(rows=1 << 24, cols=65536, x_stride=65536), -1),
    (dict(rows=1 << 24, cols=1024, x_stride=1024), -1), (dict(codes=PTR + 256), -1), (dict(scales=PTR + 1), -1),
    (dict(scales=(2 << 20) + 5), -1),
], ids=str)
def test_rounding_refuses(qm, change, code):
    a = dict(x=PTR, dtype=1, x_stride=64, rows=8, cols=64, codes=2 << 20, scales=3 << 20)
    a.update(change)
    lib = qm.library()
    _refused(qm, lib.strata_moe_mxfp_quantize(a["x"], a["dtype"], a["x_stride"], a["rows"], a["cols"], a["codes"],
                                              a["scales"], None), code)
    _refused(qm, lib.strata_moe_mxfp_dequantize(a["codes"], a["scales"], a["rows"], a["cols"], a["x"], a["dtype"],
                                                a["x_stride"], None), code)


def test_no_rows_is_a_no_op(qm):
    lib = qm.library()
    assert lib.strata_moe_mxfp_quantize(None, 1, 64, 0, 64, None, None, None) == 0
    assert lib.strata_moe_mxfp_dequantize(None, None, 0, 64, None, 2, 64, None) == 0
    st = qm.MxfpWeightsStruct(1, 8, 64, 0, None, 4096)
    assert lib.strata_moe_mxfp_product(None, None, 0, ctypes.byref(st), None, None, 0, None, 1, 8, None) == 0


@pytest.mark.parametrize("rows,cols,swiglu",
                         [(0, 64, 0), (65537, 64, 0), (7, 64, 1), (8, 40, 0), (8, 0, 0), (8, 64, 2)])
def test_packed_bytes_refuses(qm, rows, cols, swiglu):
    b = ctypes.c_int64()
    _refused(qm, qm.library().strata_moe_mxfp_packed_bytes(rows, cols, swiglu, ctypes.byref(b)), -1)


def test_packed_bytes(qm):
    # a multiple of 16 rows and 512 columns is held in 4.25 bits a value
    assert qm.strata_moe_mxfp_packed_bytes(2048, 2560, True) == 2048 * 2560 * 17 // 32
    # 16 rows of 32 values: 256 bytes of codes, and a group's scales
    assert qm.strata_moe_mxfp_packed_bytes(1, 32) == 256 + 256
    _refused(qm, qm.library().strata_moe_mxfp_packed_bytes(8, 64, 0, None), -1)


@pytest.mark.parametrize("change", [
    dict(e0=-1), dict(e0=3, e1=2), dict(e1=1025), dict(stride=512), dict(stride=1300), dict(stride=1 << 60),
    dict(codes=None), dict(scales=None), dict(packed=None), dict(codes=PTR + 8), dict(packed=(8 << 20) + 128),
    dict(codes=8 << 20), dict(scales=(8 << 20) + 2600), dict(rows=0), dict(cols=33),
], ids=str)
def test_pack_refuses(qm, change):
    a = dict(codes=PTR, scales=2 << 20, e0=0, e1=4, rows=8, cols=64, swiglu=0, packed=8 << 20, stride=1280)
    a.update(change)
    _refused(qm, qm.library().strata_moe_mxfp_pack(*a.values(), None), -1)


@pytest.mark.parametrize("change,code", [
    (dict(weights=None), -1), (dict(E=0), -1), (dict(E=1025), -1), (dict(n=0), -1), (dict(cols=72), -1),
    (dict(swiglu=3), -1), (dict(n=7, swiglu=1), -1), (dict(stride=512), -1), (dict(stride=1281), -1),
    (dict(stride=1 << 60), -1), (dict(rows=-1), -1), (dict(rows=(1 << 24) + 1), -1), (dict(x_rows=-1), -1),
    (dict(x_rows=(1 << 24) + 1, src=7 << 20), -1), (dict(dtype=9), -2), (dict(out_stride=7), -1),
    (dict(offsets=None), -1), (dict(rows=21), -1), (dict(x_rows=0, src=7 << 20), -1),
    (dict(x_rows=1 << 24, cols=512, stride=5120, src=7 << 20), -1), (dict(codes=None), -1), (dict(scales=None), -1),
    (dict(packed=None), -1), (dict(out=None), -1), (dict(codes=PTR + 4), -1), (dict(packed=(3 << 20) + 64), -1),
    (dict(offsets=(5 << 20) + 2), -1), (dict(src=(7 << 20) + 1), -1), (dict(out=(6 << 20) + 2), -1),
    (dict(out=PTR + 32), -1), (dict(out=3 << 20), -1), (dict(out=(5 << 20) - 4), -1), (dict(out=(2 << 20) + 4), -1),
    (dict(src=6 << 20), -1),
], ids=str)
def test_product_refuses(qm, change, code):
    a = dict(codes=PTR, scales=2 << 20, x_rows=20, E=4, n=8, cols=64, swiglu=0, packed=3 << 20, stride=1280,
             offsets=5 << 20, src=None, rows=20, out=6 << 20, dtype=1, out_stride=8, weights=True)
    a.update(change)
    st = qm.MxfpWeightsStruct(a["E"], a["n"], a["cols"], a["swiglu"], a["packed"], a["stride"])
    _refused(qm, qm.library().strata_moe_mxfp_product(
        a["codes"], a["scales"], a["x_rows"], ctypes.byref(st) if a["weights"] else None, a["offsets"], a["src"],
        a["rows"], a["out"], a["dtype"], a["out_stride"], None), code)


def test_the_binding_checks_its_tensors(qm):
    x = torch.zeros((4, 64))
    with pytest.raises(TypeError):
        qm.strata_moe_mxfp_quantize(x)                      # not on the GPU
    with pytest.raises(TypeError):
        qm.strata_moe_mxfp_quantize(x.int())
    with pytest.raises(ValueError):
        qm.strata_moe_mxfp_quantize(x[0])
    with pytest.raises(ValueError):
        qm.strata_moe_mxfp_quantize(x.t())
    with pytest.raises(ValueError):
        qm.strata_moe_mxfp_quantize(torch.zeros(1, 64).expand(4, 64))
    codes, scales = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    with pytest.raises(TypeError):
        qm.strata_moe_mxfp_dequantize(codes.int(), scales, x)
    with pytest.raises(ValueError):
        qm.strata_moe_mxfp_dequantize(codes[:3], scales, x)
    with pytest.raises(ValueError):
        qm.strata_moe_mxfp_dequantize(codes, scales[:, :1], x)
    with pytest.raises(ValueError):
        qm.MxfpWeights(0, 8, 64, device="cpu")
    with pytest.raises(qm.StrataMoeError):
        qm.MxfpWeights(1, 8, 65, device="cpu")
    w = qm.MxfpWeights(2, 8, 64, device="cpu")
    wc, ws = torch.zeros((2, 8, 32), dtype=torch.uint8), torch.zeros((2, 8, 2), dtype=torch.uint8)
    with pytest.raises(TypeError):
        w.pack(0, wc, ws)                                   # not on the GPU
    with pytest.raises(ValueError):
        w.pack(0, wc[:, :4], ws)
    out = torch.zeros((4, 8))
    with pytest.raises(TypeError):
        qm.strata_moe_mxfp_product(codes, scales, None, out)
    with pytest.raises(ValueError):
        qm.strata_moe_mxfp_product(codes, scales, w, out[:, :7])
    with pytest.raises(ValueError):
        qm.strata_moe_mxfp_product(codes, scales, w, out, offsets=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        qm.strata_moe_mxfp_product(codes, scales, w, out, offsets=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        qm.strata_moe_mxfp_product(codes, scales, w, out, offsets=torch.zeros(3, dtype=torch.int32),
                                   src=torch.zeros(5, dtype=torch.int32))


# ----------------------------------------------------- the reference's pins
def test_reference_rounding_by_brute_force():
    """Nearest of all 16 values in exact rationals, on a grid through every border."""
    from fractions import Fraction as F

    grid = np.arange(-33, 34) / 4.0
    for base in (4.0, 5.5, 7.75):
        vals = grid[np.abs(grid) <= base]
        for i in range(0, len(vals), 31):
            x = np.zeros((1, 32))
            x[0, :len(vals[i:i + 31])] = vals[i:i + 31]
            x[0, 31] = base
            codes, byte = ref.quantize(x)
            assert byte[0, 0] == 127
            for v, c in zip(x[0], codes[0]):
                mags = [F(m) for m in ref.MAGNITUDES.tolist()]
                a = min(F(abs(float(v))), F(6))
                best = min(range(8), key=lambda k: (abs(a - mags[k]), k % 2))
                assert (c & 7) == best and (c >> 3) == np.signbit(v)
    assert np.array_equal(ref.unpack(ref.pack(codes)), codes)
