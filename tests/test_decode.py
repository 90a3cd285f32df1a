"""The layer for a few tokens (strata_moe_decode) against the CPU oracle.

The H codes of this path are those of exact sums, so an output differs from
the oracle's only by: the routing weight's rounding to fp32, the weighted
row's, and at most Kg - 1 fp32 additions of the combine, each at most 2^-24
of the sum of absolute terms.  With one more for the second-order terms:
    |dy[t, j]| <= (Kg + 2) 2^-24 sum_k p[t,k] |D[t,k,j]|.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import synthetic as S
from layers import canonical_expert, getter, gpu_experts, rel_err, shared_args


@pytest.fixture(scope="module")
def qm():
    import quantized_routed_expert_logits_amd as qm
    return qm


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _bound(s, ref):
    """(Kg + 2) 2^-24 sum p |D| from an oracle.layer result."""
    rows = np.abs(ref["D"])[ref["slot"]].reshape(s.T, s.K, s.H)
    b = np.einsum("tk,tkh->th", ref["p"], rows)
    kg = s.K
    if ref["shared"] is not None:
        b = b + ref["shared"]["g"][:, None] * np.abs(ref["shared"]["D"])
        kg += 1
    return (kg + 2) * 2.0 ** -24 * b


def _check(s, y, ref):
    err = np.abs(y.cpu().numpy().astype(np.float64) - ref["y"])
    assert np.all(err <= _bound(s, ref) + 1e-300), f"worst {np.max(err / (_bound(s, ref) + 1e-300)):.2f} of the bound"


def _oracle(s, x, wr, bias=None):
    return oracle.layer(x, wr, bias, getter(s), s.E, s.K, fmt=s.fmt, shared=shared_args(s))


SIZES = [
    S.custom(T=1, H=128, E=1, K=1, I=64),                                 # the smallest layer
    S.custom(T=1, H=256, E=16, K=2, I=128),
    S.custom(T=64, H=256, E=16, K=2, I=128),                              # 8 rows an expert
    S.custom(T=64, H=128, E=2, K=2, I=64, shared=True),                   # every expert gets every row
    S.custom(T=63, H=384, E=70, K=5, I=192, fmt="q2_0"),                  # odd counts, a partial group of experts
    S.custom(T=7, H=640, E=65, K=16, I=320, shared=False),
    S.custom(T=13, H=512, E=6, K=2, I=640, fmt="q2_0", shared=True),
    S.custom(T=33, H=512, E=6, K=2, I=640, fmt="q2_0", shared=True),
    S.custom(T=40, H=256, E=31, K=15, I=64, skewed=True, shared=True),    # n = 640 pairs, hot experts
    S.custom(T=5, H=1280, E=12, K=3, I=448),
    S.custom(T=4, H=512, E=6, K=2, I=640, fmt="q2_0", shared=True),       # few pairs
    S.custom(T=5, H=512, E=6, K=2, I=640, fmt="q2_0", shared=True),       # one token more
    S.custom(T=16, H=768, E=129, K=9, I=256, skewed=True),                # three groups of logits, one of one expert
    S.custom(T=3, H=4096, E=3, K=1, I=64),                                # the widest hidden size
    S.custom(T=9, H=4096, E=3, K=2, I=128, shared=True),
    S.custom(T=2, H=128, E=3, K=2, I=4096),                               # the widest FFN
    S.custom(T=64, H=128, E=1024, K=16, I=64),                            # the most experts and pairs
    S.custom(T=64, H=128, E=1023, K=15, I=64, shared=True),
]


# layers whose weights are large enough for the pairs to be grouped by expert
GROUPED = [
    S.custom(T=5, H=4096, E=8, K=3, I=2048),                              # few rows of large experts
    S.custom(T=64, H=1280, E=12, K=3, I=448),                             # about 16 rows an expert
    S.custom(T=63, H=640, E=40, K=8, I=1024, skewed=True, fmt="q2_0"),
    S.custom(T=37, H=896, E=9, K=4, I=1088, shared=True),                 # chunks of every length up to 8
    S.custom(T=64, H=2048, E=2, K=2, I=256, fmt="q2_0", shared=True),     # every expert gets every row
    S.custom(T=64, H=256, E=1023, K=15, I=384, shared=True),              # the most experts and pairs
    S.custom(T=17, H=4096, E=3, K=1, I=4096),                             # the widest layer
    # either side of the choice between the two forms
    S.custom(T=32, H=1280, E=60, K=4, I=512),
    S.custom(T=33, H=1280, E=60, K=4, I=512),
]


@pytest.mark.gpu
@pytest.mark.parametrize("s", GROUPED, ids=lambda s: s.name)
def test_grouped_layer_against_the_oracle(qm, s):
    x, wr, bias = S.activations(s), S.router_weight(s), S.router_bias(s)
    ex = gpu_experts(s)
    xg, wg = _t(x), _t(wr)
    y = qm.strata_moe_decode(xg, wg, ex, s.K, torch.full_like(xg, float("nan")))
    _check(s, y, _oracle(s, x, wr, bias))
    assert torch.equal(qm.strata_moe_decode(xg, wg, ex, s.K, torch.empty_like(xg)), y)


@pytest.mark.gpu
@pytest.mark.parametrize("s", SIZES, ids=lambda s: s.name)
def test_layer_against_the_oracle(qm, s):
    x, wr, bias = S.activations(s), S.router_weight(s), S.router_bias(s)
    y = qm.strata_moe_decode(_t(x), _t(wr), gpu_experts(s), s.K, torch.full((s.T, s.H), float("nan"), device="cuda"))
    _check(s, y, _oracle(s, x, wr, bias))


@pytest.mark.gpu
def test_grouped_layer_replayed_and_at_once(qm):
    """The grouped form: equal logits (hot experts, ties), tokens that are not
    finite beside others, any workspace contents, a graph replayed between
    eager calls, two streams at once."""
    s = S.custom(T=64, H=1280, E=12, K=3, I=448)
    x, wr, ex = S.activations(s), S.router_weight(s), gpu_experts(s)
    zero = np.zeros_like(wr)
    y = qm.strata_moe_decode(_t(x), _t(zero), ex, s.K, torch.empty((s.T, s.H), device="cuda"))
    ref = _oracle(s, x, zero)
    assert np.all(ref["ids"] == [0, 1, 2])
    _check(s, y, ref)
    xg, wg = _t(x), _t(wr)
    good = qm.strata_moe_decode(xg, wg, ex, s.K, torch.empty_like(xg))
    need = qm.strata_moe_decode_workspace_bytes(s.T, s.K, ex)
    for fill in (0x00, 0xff, 0x7f):
        ws = torch.full((need + 1024,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(qm.strata_moe_decode(xg, wg, ex, s.K, torch.empty_like(xg), workspace=ws[:need]), good)
        assert torch.all(ws[need:] == fill)
    bad = xg.clone()
    bad[4, 7], bad[60, 3] = float("nan"), float("inf")
    y = qm.strata_moe_decode(bad, wg, ex, s.K, torch.empty_like(xg))
    keep = [t for t in range(s.T) if t not in (4, 60)]
    assert torch.equal(y[keep], good[keep])
    # captured, replayed with other inputs between eager calls
    xin, out = xg.clone(), torch.empty_like(xg)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qm.strata_moe_decode(xin, wg, ex, s.K, out)
    for i in range(4):
        xin.copy_(torch.roll(xg, i, 0))
        want = qm.strata_moe_decode(xin, wg, ex, s.K, torch.empty_like(xg))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.full_like(xg, float("nan")) for _ in range(8)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(8):
        for st, o in zip(streams, outs):
            qm.strata_moe_decode(xg, wg, ex, s.K, o[i], stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, good) for o2 in outs for o in o2)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 4, 9, 17, 32, 64])
def test_production_layer_sampled(qm, T):
    s = S.custom(T=T, H=2560, E=512, K=10, I=1024)
    x, wr = S.activations(s), S.router_weight(s)
    ex = gpu_experts(S.shape("window_32"))
    y = qm.strata_moe_decode(_t(x), _t(wr), ex, s.K, torch.empty((T, s.H), device="cuda")).cpu().numpy()
    tokens = sorted({0, T // 2, T - 1})
    ref = oracle.layer_tokens(x, wr, None, getter(s), s.K, tokens)
    bound = (s.K + 2) * 2.0 ** -24 * np.einsum("tk,tkh->th", ref["p"], np.abs(ref["D"]))
    assert np.all(np.abs(y[tokens] - ref["y"]) <= bound)
    # the prompt path's layer on the same tokens: other H codes at rounding ties only
    yp = qm.strata_moe_prefill(_t(x), _t(wr), ex, s.K, torch.empty((T, s.H), device="cuda")).cpu().numpy()
    assert rel_err(y, yp) <= 2e-3


@pytest.mark.gpu
def test_every_token_to_the_same_experts(qm):
    s = S.custom(T=64, H=256, E=16, K=2, I=128)
    x, wr = S.activations(s), S.router_weight(s)
    bias = np.zeros(s.E, np.float32)
    bias[[3, 11]] = 1e4
    y = qm.strata_moe_decode(_t(x), _t(wr), gpu_experts(s).with_router_bias(_t(bias)), s.K,
                             torch.empty((s.T, s.H), device="cuda"))
    _check(s, y, _oracle(s, x, wr, bias))


@pytest.mark.gpu
def test_equal_logits_zero_rows_and_tiny_values(qm):
    s = S.custom(T=5, H=256, E=16, K=2, I=128)
    x, wr = S.activations(s), np.zeros((s.H, s.E), np.float32)   # every logit equal: the first K experts
    x[1] = 0.0                                                   # every code zero
    x[2] *= np.float32(1e-30)
    x[3, 32:64] = np.float32(1e-41)                              # a subnormal block
    x[4, :32] = np.float32(np.arange(32) - 15.5)                 # quotients on a rounding tie
    x[4, 0] = 127.0
    y = qm.strata_moe_decode(_t(x), _t(wr), gpu_experts(s), s.K, torch.empty((s.T, s.H), device="cuda"))
    ref = _oracle(s, x, wr)
    assert np.all(ref["ids"] == [0, 1])
    err = np.abs(y.cpu().numpy() - ref["y"])
    assert np.all(err <= _bound(s, ref) + 2.0 ** -148)  # an fp32 subnormal's own spacing
    assert np.all(y[1].cpu().numpy() == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 6])
def test_ties_over_many_experts(qm, T):
    """Equal logits across the groups of 64 that the top-K takes at a time:
    every expert equal, and columns that come in equal pairs far apart."""
    s = S.custom(T=T, H=128, E=300, K=12, I=64)
    x, ex = S.activations(s), gpu_experts(s)
    for wr in (np.zeros((s.H, s.E), np.float32), np.tile(S.router_weight(s)[:, :150], (1, 2))):
        y = qm.strata_moe_decode(_t(x), _t(wr), ex, s.K, torch.empty((s.T, s.H), device="cuda"))
        _check(s, y, _oracle(s, x, wr))


@pytest.mark.gpu
def test_a_token_that_is_not_finite_leaves_the_others(qm):
    s = S.custom(T=9, H=256, E=16, K=2, I=128, shared=True)
    x, wr = S.activations(s), S.router_weight(s)
    ex = gpu_experts(s)
    good = qm.strata_moe_decode(_t(x), _t(wr), ex, s.K, torch.empty((s.T, s.H), device="cuda"))
    x[4, 7], x[6, 3] = np.nan, np.inf
    y = qm.strata_moe_decode(_t(x), _t(wr), ex, s.K, torch.empty((s.T, s.H), device="cuda"))
    keep = [t for t in range(s.T) if t not in (4, 6)]
    assert torch.equal(y[keep], good[keep])


@pytest.mark.gpu
def test_workspace_contents_and_bounds(qm):
    """An uninitialised workspace of just the bytes asked for, an output with
    guard rows behind it, the same bits every time."""
    s = S.custom(T=33, H=512, E=6, K=2, I=640, fmt="q2_0", shared=True)
    x, wr, ex = _t(S.activations(s)), _t(S.router_weight(s)), gpu_experts(s)
    need = qm.strata_moe_decode_workspace_bytes(s.T, s.K, ex)
    ref = None
    for fill in (0x00, 0xff, 0x7f):
        ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
        buf = torch.full((s.T + 2, s.H), 7.0, device="cuda")
        y = qm.strata_moe_decode(x, wr, ex, s.K, buf[:s.T], workspace=ws[:need])
        assert torch.all(buf[s.T:] == 7.0) and torch.all(ws[need:] == fill)
        ref = y.clone() if ref is None else ref
        assert torch.equal(y, ref)
    with pytest.raises(qm.StrataMoeError) as ei:
        qm.strata_moe_decode(x, wr, ex, s.K, torch.empty_like(x), workspace=ws[:need - 256])
    assert ei.value.code == qm.ENOMEM


@pytest.mark.gpu
def test_calls_on_two_streams_at_once(qm):
    shapes = [S.custom(T=64, H=256, E=16, K=2, I=128), S.custom(T=33, H=512, E=6, K=2, I=640, fmt="q2_0", shared=True)]
    ins = [(_t(S.activations(s)), _t(S.router_weight(s)), gpu_experts(s)) for s in shapes]
    refs = [qm.strata_moe_decode(x, wr, ex, s.K, torch.empty_like(x)) for s, (x, wr, ex) in zip(shapes, ins)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.full_like(x, float("nan")) for _ in range(20)] for x, _, _ in ins]
    torch.cuda.synchronize()
    for i in range(20):
        for j, (s, (x, wr, ex)) in enumerate(zip(shapes, ins)):
            qm.strata_moe_decode(x, wr, ex, s.K, outs[j][i], stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(o, refs[j]) for o in outs[j])


@pytest.mark.gpu
@pytest.mark.parametrize("s", [S.custom(T=1, H=256, E=16, K=2, I=128),
                               S.custom(T=33, H=512, E=6, K=2, I=640, fmt="q2_0", shared=True)], ids=lambda s: s.name)
def test_captured_and_replayed(qm, s):
    x, wr, ex = _t(S.activations(s)), _t(S.router_weight(s)), gpu_experts(s)
    out = torch.empty_like(x)
    qm.strata_moe_decode(x, wr, ex, s.K, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qm.strata_moe_decode(x, wr, ex, s.K, out)
    for i in range(4):  # new inputs in the captured buffers, eager calls in between
        x.copy_(_t(S.activations(s, seed=i + 1)))
        ref = qm.strata_moe_decode(x, wr, ex, s.K, torch.empty_like(x))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


@pytest.mark.gpu
def test_adapters_beside_the_layer(qm):
    """With adapters the call is the layer, then the adapters on its output;
    a prompt through strata_moe_prefill and strata_moe_adapt agrees."""
    s = S.custom(T=19, H=256, E=16, K=2, I=128, shared=True)
    x, wr, ex = _t(S.activations(s)), _t(S.router_weight(s)), gpu_experts(s)
    rng = torch.Generator().manual_seed(3)
    ad = qm.Adapters(torch.randn((4, 8, s.H), generator=rng).cuda().bfloat16() / 16,
                     torch.randn((4, s.H, 8), generator=rng).cuda().bfloat16(),
                     scale=torch.rand(4, generator=rng).cuda())
    ids = torch.randint(-1, 4, (s.T,), generator=rng, dtype=torch.int32).cuda()
    y = qm.strata_moe_decode(x, wr, ex, s.K, torch.empty_like(x), adapters=ad, adapter_ids=ids)
    plain = qm.strata_moe_decode(x, wr, ex, s.K, torch.empty_like(x))
    assert torch.equal(y, qm.strata_moe_adapt(x, ids, ad, plain, torch.empty_like(x)))
    assert torch.equal(y[ids < 0], plain[ids < 0]) and not torch.equal(y, plain)
    p = qm.strata_moe_prefill(x, wr, ex, s.K, torch.empty_like(x))
    qm.strata_moe_adapt(x, ids, ad, p, p)
    assert rel_err(y.cpu().numpy(), p.cpu().numpy()) <= 2e-3
    # captured, with other requests in each replay
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qm.strata_moe_decode(x, wr, ex, s.K, out, adapters=ad, adapter_ids=ids)
    for i in range(3):
        ids.copy_(torch.randint(-1, 4, (s.T,), generator=rng, dtype=torch.int32).cuda())
        ref = qm.strata_moe_decode(x, wr, ex, s.K, torch.empty_like(x), adapters=ad, adapter_ids=ids)
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


@pytest.mark.gpu
def test_a_decode_loop_on_a_stream_of_its_own(qm):
    """Calls one after another on one stream and one workspace, each on the
    output of the last, beside other work on the default stream."""
    s = S.custom(T=8, H=256, E=16, K=2, I=128)
    wr, ex = _t(S.router_weight(s)), gpu_experts(s)

    def loop(stream):
        with torch.cuda.stream(stream):
            x = _t(S.activations(s))
            ws = torch.empty(qm.strata_moe_decode_workspace_bytes(s.T, s.K, ex), dtype=torch.uint8, device="cuda")
            for _ in range(6):
                y = qm.strata_moe_decode(x, wr, ex, s.K, torch.empty_like(x), workspace=ws)
                x = y / y.abs().amax(1, keepdim=True)
        return x

    ref = loop(torch.cuda.current_stream())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    busy = torch.randn((2048, 2048), device="cuda")
    for _ in range(20):
        busy = torch.tanh(busy @ busy / 64)
    y = loop(side)
    torch.cuda.synchronize()
    assert torch.equal(y, ref)


def _cancelling_layer(H, I, where, fmt):
    """One expert whose first two blocks nearly cancel, and the rows for it.
    The codes add up to 4063 and 4061 (31 of 127 and a 126, 29 and three), the
    weights' codes are 3 and 0, their scales 2047/1024 (11 bits).  In the
    symmetric map the blocks are 12189 and -12183 (14 bits) times 2047/1024 / 2:
    24950883 / 1024 is a tie in 24 bits and rounds by 1 / 1024, and the two
    rounded products together miss their sum, 12282 / 1024, by 2^-12.6 of it.
    where: the products that cancel."""
    code = np.full(64, 127.0, np.float32)
    code[5], code[[33, 40, 63]] = 126, 126
    half = lambda v: np.float16(v).view(np.uint16)  # noqa: E731
    cgu, sgu = np.zeros((2 * I, H), np.uint8), np.zeros((2 * I, H // 32), np.uint16)
    cd, sd = np.zeros((H, I), np.uint8), np.zeros((H, I // 32), np.uint16)
    rng = np.random.default_rng(5)
    cgu[:, :32] = 3
    if where == "gate_up":
        sgu[:, :2] = half(2047 / 1024)
        sgu[I:, 1] = 0                       # up: the first block alone
        cd[:] = rng.integers(0, 4, cd.shape)
        sd[:] = rng.uniform(0.005, 0.02, sd.shape).astype(np.float16).view(np.uint16)
    else:
        sgu[:I, 0] = half(2.0 ** -10)
        sgu[I:I + 64, 0] = half(code / 128)  # h follows the same pattern, in 64 columns
        cd[:, :32] = 3
        sd[:, :2] = half(2047 / 1024)

    def rows(T):
        row = np.concatenate([code, np.zeros(H - 64, np.float32)])
        return (row * 2.0 ** (np.arange(T) % 5 - 2)[:, None]).astype(np.float32)

    return S.Expert(cgu, sgu, cd, sd), rows


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q2_sym", "q2_0"])
@pytest.mark.parametrize("where", ["gate_up", "down"])
@pytest.mark.parametrize("T, H, I", [(1, 128, 64), (5, 256, 128),         # every pair on its own
                                     (17, 4096, 1280), (20, 4096, 1088)],  # chunks of 8, 4 and 1 rows
                         ids=["1", "5", "17", "20"])
def test_the_largest_block_sums(qm, T, H, I, where, fmt):
    ex, rows = _cancelling_layer(H, I, where, fmt)
    s = S.custom(T=T, H=H, E=1, K=1, I=I, fmt=fmt)
    x, wr = rows(T), np.zeros((H, 1), np.float32)
    ref = oracle.layer(x, wr, None, lambda e: ex, 1, 1, fmt=fmt)
    if fmt == "q2_sym":  # the blocks are what the construction says
        q, c = (ref["qx"], ex.codes_gu) if where == "gate_up" else (ref["qh"], ex.codes_d)
        P = ((2 * c[0, :64].astype(int) - 3) * q[0, :64].astype(int)).reshape(2, 32).sum(1)
        assert list(P) == [12189, -12183] and np.float32(P[0]) * np.float32(2047 / 1024) != P[0] * (2047 / 1024)
    packed = qm.Experts(1, H, I, fmt=fmt)
    packed.pack(0, ex.codes_gu[None], ex.scales_gu[None], ex.codes_d[None], ex.scales_d[None])
    y = qm.strata_moe_decode(_t(x), _t(wr), packed, 1, torch.empty((T, H), device="cuda"))
    # where the blocks of D cancel, both 64-bit sums (this one and the
    # oracle's) may be off by a rounding of 2^-53 per block and part
    codes = (ex.codes_d.astype(float) - oracle.code_zero(fmt)).reshape(H, -1, 32)
    P = np.einsum("obi,tbi->tob", codes, ref["qh"].astype(float).reshape(T, -1, 32))
    terms = (np.abs(P) * ex.scales_d.view(np.float16).astype(float) * ref["sh"][:, None, :].astype(float)).sum(2)
    err = np.abs(y.cpu().numpy().astype(np.float64) - ref["y"])
    assert np.all(err <= _bound(s, ref) + 4 * (I // 32 + 8) * 2.0 ** -53 * terms), "a block's product was rounded"


@pytest.mark.gpu
def test_one_workspace_for_the_largest_call(qm):
    """A workspace sized for a grouped call serves a smaller call, whose pairs
    stay on their own and take more chunks."""
    s = S.custom(T=64, H=1024, E=8, K=2, I=1024)
    x, wr, ex = _t(S.activations(s)), _t(S.router_weight(s)), gpu_experts(s)
    for most in (41, 64):
        need = qm.strata_moe_decode_workspace_bytes(most, s.K, ex)
        ws = torch.full((need + 1024,), 0x7f, dtype=torch.uint8, device="cuda")
        for T in (most, 41, 40, 7):
            ref = qm.strata_moe_decode(x[:T], wr, ex, s.K, torch.empty_like(x[:T]))
            y = qm.strata_moe_decode(x[:T], wr, ex, s.K, torch.empty_like(x[:T]), workspace=ws[:need])
            assert torch.equal(y, ref) and torch.all(ws[need:] == 0x7f)


@pytest.mark.gpu
@pytest.mark.parametrize("mask", [-np.inf, float(np.finfo(np.float32).min)])
@pytest.mark.parametrize("s", [S.custom(T=3, H=256, E=200, K=4, I=128),
                               S.custom(T=37, H=896, E=90, K=4, I=1088, shared=True)], ids=lambda s: s.name)
def test_experts_masked_by_the_bias(qm, s, mask):
    """All experts but two masked out: the rest of a token's K are masked ones,
    in the order of their logits or (all -inf) of their indexes, of weight 0."""
    x, wr = S.activations(s), S.router_weight(s)
    bias = np.full(s.E, mask, np.float32)
    bias[[s.E // 3, s.E - 2]] = 0.5
    y = qm.strata_moe_decode(_t(x), _t(wr), gpu_experts(s).with_router_bias(_t(bias)), s.K,
                             torch.empty((s.T, s.H), device="cuda"))
    ref = _oracle(s, x, wr, bias)
    assert np.all(ref["p"][:, 2:] == 0) and np.all(np.sort(ref["ids"][:, :2], 1) == [s.E // 3, s.E - 2])
    _check(s, y, ref)


# -------------------------------------------------------- refusals (no GPU)
def _struct(qm, E=16, H=256, I=128, fmt=1):
    gu, dn = qm.strata_moe_packed_bytes(H, I)
    return qm.ExpertsStruct(E, H, I, fmt, 1 << 20, gu, 1 << 30, dn, None)


def _call(qm, st, T=4, K=2, x=1 << 16, out=1 << 24, ws=1 << 28, nbytes=1 << 40, ad=None, ids=None, wr=64):
    p = ctypes.c_void_p
    return qm.library().strata_moe_decode(p(x), p(wr), None if st is None else ctypes.byref(st), T, K,
                                          None if ad is None else ctypes.byref(ad), p(ids) if ids else None, p(out),
                                          p(ws) if ws else None, nbytes, None)


def test_refusals_on_the_host(qm):
    st = _struct(qm)
    for kw in (dict(T=-1), dict(T=65), dict(K=0), dict(K=17), dict(x=None), dict(out=None), dict(wr=None),
               dict(x=(1 << 16) + 4), dict(out=(1 << 24) + 8), dict(ws=None), dict(ws=(1 << 28) + 64),
               dict(out=1 << 16), dict(out=(1 << 16) + 2048), dict(ids=64)):
        assert _call(qm, st, **kw) == qm.EINVAL, kw
        assert qm.strata_moe_last_error() != ""
    assert _call(qm, None) == qm.EINVAL
    assert _call(qm, st, nbytes=4096) == qm.ENOMEM
    assert _call(qm, _struct(qm, fmt=7)) == qm.EUNSUPPORTED
    assert _call(qm, _struct(qm, E=2), K=3) == qm.EINVAL
    assert _call(qm, st, T=0, x=None, out=None, wr=None, ws=None, nbytes=0) == 0
    ad = qm.AdaptersStruct(2, 8, 256, 256, 1, 256, 256, None, None)
    assert _call(qm, st, ad=ad) == qm.EINVAL                                          # no adapter_ids
    for bad in (qm.AdaptersStruct(2, 8, 256, 128, 1, 256, 256, None, None),          # other widths
                qm.AdaptersStruct(2, 8, 128, 256, 1, 256, 256, None, None),
                qm.AdaptersStruct(2, 8, 256, 256, 1, None, 256, None, None),
                qm.AdaptersStruct(2, 0, 256, 256, 1, 256, 256, None, None)):
        assert _call(qm, st, ad=bad, ids=64) == qm.EINVAL


def test_workspace_on_the_rows(qm):
    st = _struct(qm)
    for ws in (1 << 16, 1 << 24, (1 << 16) + 512):
        assert _call(qm, st, ws=ws) == qm.EINVAL
        assert "workspace overlaps" in qm.strata_moe_last_error()


def test_workspace_size_query(qm):
    b = ctypes.c_size_t()
    lib, st = qm.library(), _struct(qm)
    assert lib.strata_moe_decode_workspace_bytes(64, 2, ctypes.byref(st), None, ctypes.byref(b)) == 0
    plain = b.value
    assert plain % 256 == 0 and plain > 0
    ad = qm.AdaptersStruct(2, 8, 256, 256, 3, 256, 256, None, None)
    assert lib.strata_moe_decode_workspace_bytes(64, 2, ctypes.byref(st), ctypes.byref(ad), ctypes.byref(b)) == 0
    assert b.value >= plain + 64 * 8 * 4
    assert lib.strata_moe_decode_workspace_bytes(65, 2, ctypes.byref(st), None, ctypes.byref(b)) == qm.EINVAL
    assert lib.strata_moe_decode_workspace_bytes(64, 2, ctypes.byref(st), None, None) == qm.EINVAL


def test_binding_refusals(qm):
    E, H, I, T = 8, 256, 128, 4
    ex = qm.Experts(E, H, I, device="cpu")
    x, wr, out = torch.zeros((T, H)), torch.zeros((H, E)), torch.zeros((T, H))
    ad = qm.Adapters(torch.zeros((2, 4, H)), torch.zeros((2, H, 4)))
    with pytest.raises(TypeError):
        qm.strata_moe_decode(x, wr, ex, 2, out)                       # CPU tensors
    with pytest.raises(ValueError):
        qm.strata_moe_decode(torch.zeros((T, H + 1)), wr, ex, 2, out)
    with pytest.raises(TypeError):
        qm.strata_moe_decode(x.double(), wr, ex, 2, out)
    with pytest.raises((TypeError, ValueError)):
        qm.strata_moe_decode(x, wr, ex, 2, out, adapters=ad)
    assert qm.DECODE_MAX_TOKENS == 64


@pytest.mark.parametrize("H, I, E, K", [(1024, 1024, 8, 2), (1024, 1024, 8, 8), (2560, 1024, 512, 10),
                                        (2560, 640, 512, 10), (1280, 512, 60, 4), (4096, 4096, 3, 1),
                                        (128, 64, 1024, 15), (512, 640, 6, 2)])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("rank", [0, 64])
def test_workspace_sizes_never_decrease(qm, H, I, E, K, shared, rank):
    """One workspace sized for the largest batch serves every smaller one."""
    st = _struct(qm, E - shared if E == 1024 else E, H, I)
    st.shared_gate = 1 << 12 if shared else None
    ad = qm.AdaptersStruct(2, rank, H, H, 3, 256, 256, None, None)
    b, last = ctypes.c_size_t(), 0
    for T in range(65):
        assert qm.library().strata_moe_decode_workspace_bytes(
            T, K, ctypes.byref(st), ctypes.byref(ad) if rank else None, ctypes.byref(b)) == 0
        assert b.value >= last, T
        last = b.value
