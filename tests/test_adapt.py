"""Per-request low-rank adapters (strata_moe_adapt) against the definition in
64 bits: out[t] = y[t] + scale_a B_a (A_a x[t]).

Tolerance, from the arithmetic: every product of two fp32 values enters its
fp32 sum rounded once, or as at most three exact parts, and the sum has at
most 3 n + 8 roundings of 2^-24 for n products, in any order, each relative
to at most the sum of absolute terms.  So with u = 2^-24, absolute values
throughout and V = |A| |x|:
    |dv|   <= (3 in + 8) u V
    |dout| <= |scale| (|B| |dv| + (3 rank + 8) u |B| (V + |dv|))
              + 3 u (|y| + |scale| |B| V),
the last for the scaling and the addition to y (1 % on top for the products
of these factors).
"""
import ctypes

import numpy as np
import pytest
import torch

U = 2.0 ** -24


@pytest.fixture(scope="module")
def qm():
    import quantized_routed_expert_logits_amd as qm
    return qm


def _reference(x, ids, a, b, scale, ranks, y):
    """(out, tolerance) in 64 bits on the CPU."""
    x, y, a, b = (v.double().cpu().numpy() for v in (x, y, a, b))
    ids = ids.cpu().numpy()
    out, tol = y.copy(), np.zeros_like(y)
    n_in, rank = x.shape[1], a.shape[1]
    for n in range(a.shape[0]):
        rows = np.nonzero(ids == n)[0]
        r = rank if ranks is None else int(np.clip(ranks[n].item(), 0, rank))
        sc = 1.0 if scale is None else float(scale[n])
        A, B = a[n, :r], b[n, :, :r]
        out[rows] += sc * ((x[rows] @ A.T) @ B.T)
        V = np.abs(x[rows]) @ np.abs(A).T
        dv = (3 * n_in + 8) * U * V
        BV = V @ np.abs(B).T
        tol[rows] = 1.01 * (abs(sc) * (dv @ np.abs(B).T + (3 * r + 8) * U * (V + dv) @ np.abs(B).T)
                            + 3 * U * (np.abs(y[rows]) + abs(sc) * BV))
    return out, tol


def _check(out, ref):
    want, tol = ref
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= tol), f"worst {np.nanmax(err / np.maximum(tol, 1e-300)):.2f} of the tolerance"


def _case(T, n_in, n_out, rank, L, dtype, seed=0, pad=0, ids=None, layout="random"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, n_in + pad), generator=g).cuda()[:, :n_in]
    y = torch.randn((T, n_out + pad), generator=g).cuda()[:, :n_out]
    a = (torch.randn((L, rank, n_in), generator=g) / n_in ** 0.5).to(dtype).cuda()
    b = torch.randn((L, n_out, rank), generator=g).to(dtype).cuda()
    scale = (torch.rand(L, generator=g) + 0.5).cuda()
    if ids is None:
        if layout == "random":
            ids = torch.randint(-1, L, (T,), generator=g)
        else:  # runs of one request
            cuts = torch.sort(torch.randint(0, T, (min(T, 6),), generator=g)).values
            ids = torch.randint(-1, L, (7,), generator=g)[torch.searchsorted(cuts, torch.arange(T), right=True)]
    return x, ids.to(torch.int32).cuda(), a, b, scale, y


SIZES = [
    # T, in, out, rank, adapters, pad, layout
    (1, 1, 1, 1, 1, 0, "random"),
    (1, 256, 256, 8, 3, 0, "random"),
    (5, 7, 3, 2, 2, 0, "random"),
    (16, 64, 128, 16, 4, 0, "random"),
    (17, 1000, 333, 13, 5, 3, "random"),
    (33, 128, 2560, 64, 40, 0, "random"),
    (64, 2560, 512, 16, 64, 4, "random"),
    (65, 96, 80, 5, 3, 0, "runs"),
    (100, 260, 100, 100, 2, 0, "runs"),
    (130, 384, 640, 256, 3, 0, "runs"),
    (256, 100, 70, 9, 6, 0, "random"),       # the last call that spreads a tile's adapters
    (257, 100, 70, 9, 6, 0, "random"),
    (500, 33, 65, 17, 9, 5, "random"),
    (1000, 544, 200, 65, 4, 0, "runs"),      # a second run of 64 ranks, a step that ends inside it
    (1025, 512, 256, 8, 7, 0, "runs"),
    (2049, 640, 1024, 32, 6, 0, "runs"),
    (700, 2560, 2560, 64, 8, 0, "runs"),
    (5000, 48, 2564, 20, 3, 0, "runs"),      # y read past the caches, outputs that end inside a run
    (3, 65536, 5, 3, 2, 0, "random"),
    (2, 8, 65536, 4, 2, 0, "random"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
def test_against_the_definition(qm, size, dtype):
    T, n_in, n_out, rank, L, pad, layout = size
    x, ids, a, b, scale, y = _case(T, n_in, n_out, rank, L, dtype, seed=T, pad=pad, layout=layout)
    buf = torch.full((T, n_out + 3), 7.0, device="cuda")
    out = qm.strata_moe_adapt(x, ids, qm.Adapters(a, b, scale), y, buf[:, :n_out])
    _check(out, _reference(x, ids, a, b, scale, None, y))
    assert torch.all(buf[:, n_out:] == 7.0)                   # the rows' padding
    none = (ids < 0)
    assert torch.equal(out[none], y[none])
    # in place, and the same bits again
    y2 = y.clone(memory_format=torch.contiguous_format)
    qm.strata_moe_adapt(x, ids, qm.Adapters(a, b, scale), y2, y2)
    assert torch.equal(y2, out)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T", [3, 40, 300])
def test_ranks_per_adapter(qm, T, dtype):
    """Ranks of 0, odd, full and (clamped) beyond it; what lies behind an
    adapter's rank is never used, be it NaN or infinite."""
    x, _, a, b, scale, y = _case(T, 200, 136, 24, 6, dtype, seed=T)
    ids = (torch.arange(T) * 5 % 6).to(torch.int32).cuda()
    ranks = torch.tensor([0, 1, 13, 24, 99, -4], dtype=torch.int32).cuda()
    for n, r in enumerate([0, 1, 13]):
        a[n, r:], b[n, :, r:] = float("nan"), float("inf")
    a[5], b[5] = float("nan"), float("nan")  # rank -4 counts as 0
    out = qm.strata_moe_adapt(x, ids, qm.Adapters(a, b, scale, ranks), y, torch.empty_like(y))
    _check(out, _reference(x, ids, a, b, scale, ranks, y))
    empty = (ids == 0) | (ids == 5)
    assert torch.equal(out[empty], y[empty])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T, rank", [(40, 16), (40, 64), (300, 64), (40, 72)])
def test_ranks_that_end_inside_a_step(qm, T, rank, dtype):
    """Ranks at and around the steps' ends, below rows of B that go on past
    the last step: their rest is read, and none of it is used."""
    use = [r for r in (1, 7, 8, 15, 16, 31, 32, 33, 47, 63, 64, 65, 72) if r <= rank]
    x, _, a, b, scale, y = _case(T, 96, 136, rank, len(use), dtype, seed=T + rank)
    ids = (torch.arange(T) * 5 % len(use)).to(torch.int32).cuda()
    for n, r in enumerate(use):
        a[n, r:], b[n, :, r:] = float("inf"), float("nan")
    ranks = torch.tensor(use, dtype=torch.int32).cuda()
    out = qm.strata_moe_adapt(x, ids, qm.Adapters(a, b, scale, ranks), y, torch.empty_like(y))
    _check(out, _reference(x, ids, a, b, scale, ranks, y))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 31, 200])
def test_ids_outside_the_adapters_and_no_scale(qm, T):
    x, _, a, b, _, y = _case(T, 128, 72, 8, 3, torch.bfloat16, seed=1)
    ids = torch.tensor([-1, 3, 1 << 30, -(1 << 31), 2, 0])[torch.arange(T) % 6].to(torch.int32).cuda()
    out = qm.strata_moe_adapt(x, ids, qm.Adapters(a, b), y, torch.empty_like(y))
    _check(out, _reference(x, ids, a, b, None, None, y))
    outside = (ids < 0) | (ids >= 3)
    assert torch.equal(out[outside], y[outside])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [16, 48, 128])
def test_values_that_are_not_finite_stay_in_their_rows(qm, T):
    """A request whose input or adapter holds NaN or infinities changes no
    other request's row."""
    x, ids, a, b, scale, y = _case(T, 96, 160, 16, 4, torch.float16, ids=torch.arange(T) % 4)
    ad = qm.Adapters(a, b, scale)
    good = qm.strata_moe_adapt(x, ids, ad, y, torch.empty_like(y))
    a2, b2, x2 = a.clone(), b.clone(), x.clone()
    a2[1, 3, 5], b2[1, 9, 2], b2[2, 0, 0] = float("inf"), float("nan"), float("-inf")
    x2[3, 0], y2 = float("nan"), y.clone()
    y2[7, 1] = float("inf")
    out = qm.strata_moe_adapt(x2, ids, qm.Adapters(a2, b2, scale), y2, torch.empty_like(y))
    keep = [t for t in range(T) if ids[t] not in (1, 2) and t not in (3, 7)]
    assert torch.equal(out[keep], good[keep])
    assert torch.isnan(out[3]).all() and torch.isinf(out[7, 1])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 70])
def test_unaligned_bases_and_strides(qm, T):
    """Rows that start at any element, adapters at any element."""
    n_in, n_out, rank, L = 256, 128, 16, 3
    g = torch.Generator().manual_seed(5)
    x = torch.randn(T * 257 + 1, generator=g).cuda()[1:].view(T, 257)[:, :n_in]
    y = torch.randn(T * 131 + 3, generator=g).cuda()[3:].view(T, 131)[:, :n_out]
    a = torch.randn(L * rank * n_in + 1, generator=g).bfloat16().cuda()[1:].view(L, rank, n_in)
    b = torch.randn(L * rank * n_out + 3, generator=g).bfloat16().cuda()[3:].view(L, n_out, rank)
    ids = torch.randint(-1, L, (T,), generator=g, dtype=torch.int32).cuda()
    out = torch.empty(T * 129 + 1, device="cuda")[1:].view(T, 129)[:, :n_out]
    qm.strata_moe_adapt(x, ids, qm.Adapters(a, b), y, out)
    _check(out, _reference(x, ids, a, b, None, None, y))


@pytest.mark.gpu
def test_adapters_beyond_32_bit_offsets(qm):
    L, rank, n_in, n_out = 140, 256, 65536, 24  # 2.3e9 elements of A
    a = torch.zeros((L, rank, n_in), dtype=torch.float16, device="cuda")
    b = torch.zeros((L, n_out, rank), dtype=torch.float16, device="cuda")
    g = torch.Generator().manual_seed(2)
    for n in (0, L - 1):
        a[n] = (torch.randn((rank, n_in), generator=g) / 256).half().cuda()
        b[n] = torch.randn((n_out, rank), generator=g).half().cuda()
    x = torch.randn((4, n_in), generator=g).cuda()
    y = torch.randn((4, n_out), generator=g).cuda()
    ids = torch.tensor([L - 1, 0, L - 1, 70], dtype=torch.int32).cuda()
    out = qm.strata_moe_adapt(x, ids, qm.Adapters(a, b), y, torch.empty_like(y))
    small = torch.tensor([1, 0, 1, -1], dtype=torch.int32)
    _check(out, _reference(x, small, a[[0, L - 1]], b[[0, L - 1]], None, None, y))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 24, 400])
def test_captured_and_replayed_with_other_ids(qm, T):
    x, ids, a, b, scale, y = _case(T, 320, 192, 16, 5, torch.bfloat16, seed=9)
    ad, out = qm.Adapters(a, b, scale), torch.empty_like(y)
    qm.strata_moe_adapt(x, ids, ad, y, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qm.strata_moe_adapt(x, ids, ad, y, out)
    for i in range(4):
        g = torch.Generator().manual_seed(i)
        ids.copy_(torch.randint(-1, 5, (T,), generator=g, dtype=torch.int32).cuda())
        x.copy_(torch.randn(x.shape, generator=g).cuda())
        ref = qm.strata_moe_adapt(x, ids, ad, y, torch.empty_like(y))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


@pytest.mark.gpu
def test_beside_the_router_on_two_streams(qm):
    """The adapters beside the router's projection, and calls on two streams
    at once, each with a workspace of its own."""
    cases = [_case(48, 256, 16, 8, 4, torch.float32, seed=1), _case(700, 512, 256, 16, 4, torch.bfloat16, seed=2)]
    ads = [qm.Adapters(c[2], c[3], c[4]) for c in cases]
    refs = [qm.strata_moe_adapt(c[0], c[1], ad, c[5], torch.empty_like(c[5])) for c, ad in zip(cases, ads)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.full_like(c[5], float("nan")) for _ in range(20)] for c in cases]
    torch.cuda.synchronize()
    for i in range(20):
        for j, (c, ad) in enumerate(zip(cases, ads)):
            qm.strata_moe_adapt(c[0], c[1], ad, c[5], outs[j][i], stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(o, refs[j]) for o in outs[j])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 70])
def test_columns_of_one_array(qm, T):
    """x, y and out as neighbouring columns of one buffer; what is beside them
    stays as it was."""
    x, ids, a, b, scale, y = _case(T, 64, 48, 16, 4, torch.float32, seed=6)
    ad = qm.Adapters(a, b, scale)
    ref = qm.strata_moe_adapt(x, ids, ad, y, torch.empty_like(y))
    buf = torch.full((T, 48 + 64 + 48 + 5), 7.0, device="cuda")
    out, xc, yc = buf[:, :48], buf[:, 48:112], buf[:, 112:160]
    xc.copy_(x)
    yc.copy_(y)
    qm.strata_moe_adapt(xc, ids, ad, yc, out)
    assert torch.equal(out, ref) and torch.equal(xc, x) and torch.equal(yc, y) and torch.all(buf[:, 160:] == 7.0)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 70])
def test_columns_of_one_array(qm, T):
    """x, y and out as neighbouring columns of one buffer; what is beside them
    stays as it was."""
    x, ids, a, b, scale, y = _case(T, 64, 48, 16, 4, torch.float32, seed=6)
    ad = qm.Adapters(a, b, scale)
    ref = qm.strata_moe_adapt(x, ids, ad, y, torch.empty_like(y))
    buf = torch.full((T, 48 + 64 + 48 + 5), 7.0, device="cuda")
    out, xc, yc = buf[:, :48], buf[:, 48:112], buf[:, 112:160]
    xc.copy_(x)
    yc.copy_(y)
    qm.strata_moe_adapt(xc, ids, ad, yc, out)
    assert torch.equal(out, ref) and torch.equal(xc, x) and torch.equal(yc, y) and torch.all(buf[:, 160:] == 7.0)


@pytest.mark.gpu
def test_workspace_contents_and_size(qm):
    x, ids, a, b, scale, y = _case(77, 320, 192, 16, 5, torch.float16, seed=4)
    ad = qm.Adapters(a, b, scale)
    need = qm.strata_moe_adapt_workspace_bytes(77, ad)
    ref = qm.strata_moe_adapt(x, ids, ad, y, torch.empty_like(y))
    for fill in (0x00, 0xff, 0x7f):
        ws = torch.full((need + 1024,), fill, dtype=torch.uint8, device="cuda")
        out = qm.strata_moe_adapt(x, ids, ad, y, torch.empty_like(y), workspace=ws[:need])
        assert torch.equal(out, ref) and torch.all(ws[need:] == fill)
    with pytest.raises(qm.StrataMoeError) as ei:
        qm.strata_moe_adapt(x, ids, ad, y, out, workspace=ws[:need - 256])
    assert ei.value.code == qm.ENOMEM
    e = qm.strata_moe_adapt(x[:0], ids[:0], ad, y[:0], out[:0])  # no tokens
    assert e.shape == (0, 192)


@pytest.mark.gpu
def test_one_workspace_for_the_largest_call(qm):
    """A workspace sized for many tokens serves calls of fewer, which split the
    reduction further, and is not written past its end."""
    x, ids, a, b, scale, y = _case(4097, 2560, 40, 64, 5, torch.bfloat16, seed=8, layout="runs")
    ad = qm.Adapters(a, b, scale)
    need = qm.strata_moe_adapt_workspace_bytes(4097, ad)
    ws = torch.full((need + 1024,), 0x7f, dtype=torch.uint8, device="cuda")
    for T in (4097, 4096, 2048, 257, 256, 103, 102, 1):
        ref = qm.strata_moe_adapt(x[:T], ids[:T], ad, y[:T], torch.empty_like(y[:T]))
        out = qm.strata_moe_adapt(x[:T], ids[:T], ad, y[:T], torch.empty_like(y[:T]), workspace=ws[:need])
        assert torch.equal(out, ref) and torch.all(ws[need:] == 0x7f)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T, rank", [(1, 1), (40, 1), (40, 16), (40, 64), (300, 24)])
def test_infinities_are_those_of_the_definition(qm, T, rank, dtype):
    """Infinite inputs and weights, also beside zeros and values that bf16
    holds whole: an infinity where 64 bits give one, NaN where they give NaN."""
    x, ids, a, b, scale, y = _case(T, 96, 160, rank, 4, dtype, seed=T + rank, ids=torch.arange(T) % 4)
    inf = float("inf")
    a[0, :, 5], b[0, 0::2], b[0, 1::2] = 0.5, 0.25, -0.25
    x[0::8, 5] = inf                          # adapter 0: +-inf in every column
    a[0, 0, 6] = 0.0
    x[4::8, 6] = -inf                         # adapter 0: 0 inf in the first rank, so NaN
    b[1, 9, rank // 2] = inf
    a[2, rank - 1, 7], b[2, 11] = -inf, 0.0   # adapter 2: infinite but for 0 inf in column 11
    x[0::3, 7] = x[0::3, 7].bfloat16().float()
    x[3::8, 50] = float("nan")
    y[1::2, 3] = inf
    with np.errstate(invalid="ignore"):
        want, _ = _reference(x, ids, a, b, scale, None, y)
    out = qm.strata_moe_adapt(x, ids, qm.Adapters(a, b, scale), y, torch.empty_like(y)).cpu().numpy()
    assert np.isinf(want).any() and (T < 8 or np.isnan(want).any())
    assert np.array_equal(np.isnan(out), np.isnan(want))
    assert np.array_equal(out[np.isinf(want)], want[np.isinf(want)].astype(np.float32))
    assert np.array_equal(np.isfinite(out), np.isfinite(want))


# -------------------------------------------------------- refusals (no GPU)
def _call(qm, ad, T=4, x=1 << 20, xs=256, ids=64, y=1 << 24, ys=128, out=1 << 26, os_=128, ws=1 << 28, n=1 << 40):
    p = ctypes.c_void_p
    return qm.library().strata_moe_adapt(p(x), xs, p(ids), None if ad is None else ctypes.byref(ad), T, p(y), ys,
                                         p(out), os_, p(ws) if ws else None, n, None)


def _ad(qm, L=2, rank=8, n_in=256, n_out=128, dtype=1, a=256, b=256, scale=None, ranks=None):
    return qm.AdaptersStruct(L, rank, n_in, n_out, dtype, a, b, scale, ranks)


def test_refusals_on_the_host(qm):
    for kw in (dict(L=0), dict(L=65537), dict(rank=0), dict(rank=257), dict(n_in=0), dict(n_out=65537), dict(a=None),
               dict(b=None), dict(a=258), dict(dtype=3, b=257), dict(scale=66), dict(ranks=65)):
        assert _call(qm, _ad(qm, **kw)) == qm.EINVAL, kw
        assert qm.strata_moe_last_error() != ""
    assert _call(qm, _ad(qm, dtype=9)) == qm.EUNSUPPORTED
    assert _call(qm, None) == qm.EINVAL
    good = _ad(qm)
    for kw in (dict(T=-1), dict(T=(1 << 24) + 1), dict(xs=255), dict(ys=127), dict(os_=127), dict(xs=1 << 33),
               dict(x=None), dict(ids=None), dict(y=None), dict(out=None), dict(x=(1 << 20) + 2),
               dict(out=(1 << 26) + 1), dict(ws=None), dict(ws=(1 << 28) + 128),
               dict(out=1 << 20),                      # out on x
               dict(out=(1 << 24) + 512),              # out inside y
               dict(out=1 << 24, os_=129)):            # y's memory, other rows
        assert _call(qm, good, **kw) == qm.EINVAL, kw
    assert _call(qm, good, n=64) == qm.ENOMEM
    assert _call(qm, good, T=0, x=None, ids=None, y=None, out=None, ws=None, n=0) == 0
    b = ctypes.c_size_t()
    assert qm.library().strata_moe_adapt_workspace_bytes(4, ctypes.byref(good), None) == qm.EINVAL
    assert qm.library().strata_moe_adapt_workspace_bytes(1000, ctypes.byref(good), ctypes.byref(b)) == 0
    assert b.value >= 1000 * 8 * 4


def test_binding_refusals(qm):
    a, b = torch.zeros((2, 4, 16)), torch.zeros((2, 8, 4))
    for aa, bb in ((a[0], b), (a, b[0]), (a, torch.zeros((3, 8, 4))), (a, torch.zeros((2, 8, 5))),
                   (a.transpose(1, 2), torch.zeros((2, 8, 16)))):
        with pytest.raises(ValueError):
            qm.Adapters(aa, bb)
    for aa, bb in ((a.double(), b.double()), (a, b.half())):
        with pytest.raises(TypeError):
            qm.Adapters(aa, bb)
    with pytest.raises(ValueError):
        qm.Adapters(a, b, scale=torch.zeros(3))
    with pytest.raises(TypeError):
        qm.Adapters(a, b, ranks=torch.zeros(2))
    ad = qm.Adapters(a, b)
    x, y, ids = torch.zeros((3, 16)), torch.zeros((3, 8)), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        qm.strata_moe_adapt(x, ids, ad, y, y)  # CPU tensors
    for xx, ii, yy, oo in ((torch.zeros((3, 15)), ids, y, y), (x, ids[:2], y, y), (x, ids, y[:2], y),
                           (x, ids, y, torch.zeros((8, 3)).T), (x[:, ::2], ids, y, y),
                           (x, ids, torch.zeros(1, 8).expand(3, 8), y)):
        with pytest.raises(ValueError):
            qm.strata_moe_adapt(xx, ii, ad, yy, oo)
    with pytest.raises(TypeError):
        qm.strata_moe_adapt(x, ids.long(), ad, y, y)


def test_overlaps(qm):
    """Rows of one stride beside each other do not overlap (such a call gets as
    far as the workspace's size), whatever comes first; rows that share an
    element do."""
    ad = _ad(qm, n_in=24, n_out=16)
    base, s = 1 << 24, 100

    def code(xc, yc, oc, strides=(s, s, s), T=4, ws=1 << 28, n=1):
        return _call(qm, ad, T=T, x=base + 4 * xc, xs=strides[0], y=base + 4 * yc, ys=strides[1], out=base + 4 * oc,
                     os_=strides[2], ws=ws, n=n)

    for xc, yc, oc in ((0, 24, 40), (16, 40, 0), (40, 0, 24), (24, 84, 300), (0, 24, 24), (60, 44, 84), (60, 44, 184),
                       (76, 160, 60), (400, 84, 284)):
        assert code(xc, yc, oc) == qm.ENOMEM, (xc, yc, oc)
    for xc, yc, oc in ((0, 24, 23), (0, 24, 39), (0, 24, 9), (16, 40, 1), (16, 40, 99), (0, 300, 285), (0, 40, 123),
                       (285, 0, 100)):
        assert code(xc, yc, oc) == qm.EINVAL, (xc, yc, oc)
    assert code(0, 24, 40, (s, s, s + 1)) == qm.EINVAL  # other strides: by the whole ranges
    assert code(0, 24, 40, (s, s, s + 1), T=1) == qm.ENOMEM
    assert code(0, 24, 40, ws=base, n=1 << 30) == qm.EINVAL  # the workspace on the rows
    assert code(0, 24, 40, ws=base - 256, n=1 << 30) == qm.EINVAL


def test_overlaps(qm):
    """Rows of one stride beside each other do not overlap (such a call gets as
    far as the workspace's size), whatever comes first; rows that share an
    element do."""
    ad = _ad(qm, n_in=24, n_out=16)
    base, s = 1 << 24, 100

    def code(xc, yc, oc, strides=(s, s, s), T=4, ws=1 << 28, n=1):
        return _call(qm, ad, T=T, x=base + 4 * xc, xs=strides[0], y=base + 4 * yc, ys=strides[1], out=base + 4 * oc,
                     os_=strides[2], ws=ws, n=n)

    for xc, yc, oc in ((0, 24, 40), (16, 40, 0), (40, 0, 24), (24, 84, 300), (0, 24, 24), (60, 44, 84), (60, 44, 184),
                       (76, 144, 60), (424, 84, 200), (16, 40, 99)):
        assert code(xc, yc, oc) == qm.ENOMEM, (xc, yc, oc)
    for xc, yc, oc in ((0, 24, 23), (0, 24, 39), (0, 24, 9), (16, 40, 1), (16, 40, 101), (0, 300, 285), (0, 40, 123),
                       (285, 0, 100)):
        assert code(xc, yc, oc) == qm.EINVAL, (xc, yc, oc)
    assert code(0, 24, 40, (s, s, s + 1)) == qm.EINVAL  # other strides: by the whole ranges
    assert code(0, 24, 40, (s, s, s + 1), T=1) == qm.ENOMEM
    assert code(0, 24, 40, ws=base, n=1 << 30) == qm.EINVAL  # the workspace on the rows
    assert code(0, 24, 40, ws=base + 256, n=1 << 30) == qm.EINVAL


@pytest.mark.parametrize("rank, n_in", [(64, 2560), (16, 2560), (65, 2560), (256, 2560), (1, 100), (13, 1000),
                                        (64, 513), (200, 65536), (8, 65536), (256, 9000)])
def test_workspace_sizes_never_decrease(qm, rank, n_in):
    """One workspace sized for the largest batch serves every smaller one."""
    b, lib = ctypes.c_size_t(), qm.library()
    ad = _ad(qm, rank=rank, n_in=n_in)
    last = 0
    for T in [*range(9000), *range(9000, 1 << 24, 99991)]:
        assert lib.strata_moe_adapt_workspace_bytes(T, ctypes.byref(ad), ctypes.byref(b)) == 0
        assert b.value >= last, T
        last = b.value


def test_a_workspace_that_ends_on_the_rows(qm):
    """Its first bytes lie before the rows, the last it needs on them."""
    ad = _ad(qm, n_in=24, n_out=16)
    b = ctypes.c_size_t()
    assert qm.library().strata_moe_adapt_workspace_bytes(40, ctypes.byref(ad), ctypes.byref(b)) == 0 and b.value > 256
    for rows in ("x", "y", "out"):
        at = dict(x=1 << 20, y=1 << 24, out=1 << 26)
        ws = at[rows] - 256
        assert _call(qm, ad, T=40, xs=100, ys=100, os_=100, ws=ws, n=1 << 30, **at) == qm.EINVAL
        assert "workspace overlaps" in qm.strata_moe_last_error()
