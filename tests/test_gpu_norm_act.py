"""awq_rmsnorm(_fp8) and awq_silu_mul(_fp8) against their formulas in fp64.

Tolerances, from the number formats alone:
  fp16 y   half a step, 2^-11 |y| (2^-25 among the subnormals), plus the fp32
           arithmetic: the sum of squares is a chain of at most K/1024 + 8
           terms a thread and a tree of 10 levels, so (K/1024 + 20) 2^-24; the
           inverse root, the products and the sigmoid's two special functions
           stay below 2^-20; the sigmoid's argument |g| log2(e) is rounded
           once, which moves 2^-argument by |g| 2^-24 relative.
  x8 sx    half an E4M3 step, 2^-4 |y| (sx 2^-10 among the subnormals), plus
           the same.
  h        x + residual rounded once: equal to torch's sum in fp32 rounded.
"""
import pytest
import torch

import weight_only_bit_awq_b200 as awq

pytestmark = pytest.mark.gpu

EPS = 1e-5


def fp32_slack(K):
    return (K / 1024 + 20) * 2.0 ** -24 + 2.0 ** -20


def check_fp16(y, ref, rel, what):
    err = (y.double() - ref).abs()
    lim = (2.0 ** -11 + rel) * ref.abs() + 2.0 ** -25
    assert (err <= lim).all(), (what, float((err / lim).max()))


def check_fp8(x8, sx, ref, rel, what):
    amax = ref.abs().amax(dim=1)
    assert ((sx.double() - amax / 448).abs() <= (rel + 2.0 ** -22) * amax / 448).all(), what
    got = x8.view(torch.float8_e4m3fn).double() * sx.double()[:, None]
    lim = (2.0 ** -4 + 2 * rel + 2.0 ** -20) * ref.abs() + (amax / 448 * 2.0 ** -10)[:, None]
    assert ((got - ref).abs() <= lim).all(), what
    assert (x8.view(torch.float8_e4m3fn).float().abs().amax(dim=1)[amax > 0] == 448).all(), what


def norm_ref(x, w, eps, residual=None):
    h = x.double() if residual is None else x.double() + residual.double()
    return h * (h.square().mean(dim=1, keepdim=True) + eps).rsqrt() * w.double()


def inputs(M, K, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + M * 31 + K)
    x = (torch.randn(M, K, generator=g, device="cuda") * std).half()
    r = (torch.randn(M, K, generator=g, device="cuda") * 3).half()
    w = (1 + 0.3 * torch.randn(K, generator=g, device="cuda")).half()
    return x, r, w


# rows held in registers with 1, 2 and 4 vectors per thread, and the long rows
WIDTHS = [8, 16, 120, 256, 1000, 4096, 4104, 8192, 11008, 14848, 16384, 16392, 28672, 32768, 32776, 65536]


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("M", [1, 2, 37])
@pytest.mark.parametrize("with_residual", [False, True])
def test_rmsnorm(M, K, with_residual):
    x, r, w = inputs(M, K)
    r = r if with_residual else None
    ref = norm_ref(x, w, EPS, r)
    got = awq.awq_rmsnorm(x, w, EPS, residual=r)
    y, h = got if with_residual else (got, None)
    check_fp16(y, ref, fp32_slack(K), (M, K))
    got8 = awq.awq_rmsnorm_fp8(x, w, EPS, residual=r)
    check_fp8(got8[0], got8[1], ref, fp32_slack(K), (M, K))
    if with_residual:
        want = (x.float() + r.float()).half()
        assert torch.equal(h, want) and torch.equal(got8[2], want)


def test_rmsnorm_many_rows_walk_all_rows():
    # more rows than CTAs that fit at once
    x, r, w = inputs(20011, 264)
    y, h = awq.awq_rmsnorm(x, w, EPS, residual=r)
    check_fp16(y, norm_ref(x, w, EPS, r), fp32_slack(264), "many")
    x8, sx, h8 = awq.awq_rmsnorm_fp8(x, w, EPS, residual=r)
    check_fp8(x8, sx, norm_ref(x, w, EPS, r), fp32_slack(264), "many fp8")
    assert torch.equal(h, h8)


@pytest.mark.parametrize("K", [512, 8192, 33000])
@pytest.mark.parametrize("onto", ["x", "residual"])
def test_rmsnorm_in_place(K, onto):
    x, r, w = inputs(300, K, seed=3)
    ref, want = norm_ref(x, w, EPS, r), (x.float() + r.float()).half()
    target = x if onto == "x" else r
    y, h = awq.awq_rmsnorm(x, w, EPS, residual=r, h=target)
    assert h.data_ptr() == target.data_ptr() and torch.equal(target, want)
    check_fp16(y, ref, fp32_slack(K), "in place")


def test_rmsnorm_edges():
    K = 512
    w = torch.ones(K, device="cuda").half()
    x = torch.zeros(8, K, device="cuda").half()
    x[1] = 60000.0                                # squares far beyond fp16
    x[2] = 2.0 ** -24                             # the smallest fp16: eps decides
    x[3, 7] = float("inf")
    x[4, 9] = float("nan")
    x[5, 0] = -65504.0
    x[6] = -0.0
    ok = [0, 1, 2, 5, 6, 7]
    ref = norm_ref(x, w, EPS)
    y = awq.awq_rmsnorm(x, w, EPS)
    check_fp16(y[ok], ref[ok], fp32_slack(K), "edges")
    assert (y[0] == 0).all()
    x8, sx = awq.awq_rmsnorm_fp8(x, w, EPS)
    assert (x8[0] == 0).all() and sx[0] == 0 and (x8[6] == 0).all() and sx[6] == 0
    check_fp8(x8[[1, 2, 5]], sx[[1, 2, 5]], ref[[1, 2, 5]], fp32_slack(K), "edges fp8")
    for bad in (3, 4):
        assert not torch.isfinite(y[bad]).all() and not torch.isfinite(sx[bad])
    # the sum of x and residual beyond fp16 overflows h, not y
    r = x.clone()
    y, h = awq.awq_rmsnorm(x[1:2], w, EPS, residual=r[1:2])
    assert torch.isinf(h).all()
    check_fp16(y, norm_ref(x[1:2], w, EPS, r[1:2]), fp32_slack(K), "overflowing residual")


def test_rmsnorm_without_eps_of_a_zero_row():
    x, _, w = inputs(2, 256)
    x[1] = 0
    y = awq.awq_rmsnorm(x, w, 0.0)
    check_fp16(y[:1], norm_ref(x[:1], w, 0.0), fp32_slack(256), "eps 0")
    assert torch.isnan(y[1]).all()                # 0 * (1 / 0), as the formula says


def silu_ref(gu):
    g, u = gu.double().chunk(2, dim=1)
    return g / (1 + torch.exp(-g)) * u


@pytest.mark.parametrize("F", [8, 24, 512, 1000, 4096, 4104, 11008, 14336, 16392, 28672, 32768, 32776, 65536])
@pytest.mark.parametrize("M", [1, 3, 41])
def test_silu_mul(M, F):
    g = torch.Generator(device="cuda").manual_seed(M * 100003 + F)
    gu = (torch.randn(M, 2 * F, generator=g, device="cuda") * 2).half()
    ref = silu_ref(gu)
    rel = (float(gu[:, :F].abs().max()) + 16) * 2.0 ** -23
    check_fp16(awq.awq_silu_mul(gu), ref, rel, (M, F))
    x8, sx = awq.awq_silu_mul_fp8(gu)
    check_fp8(x8, sx, ref, rel, (M, F))


def test_silu_mul_many_rows():
    gu = (torch.randn(30011, 48, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * 2).half()
    rel = 40 * 2.0 ** -23
    check_fp16(awq.awq_silu_mul(gu), silu_ref(gu), rel, "many")
    check_fp8(*awq.awq_silu_mul_fp8(gu), silu_ref(gu), rel, "many fp8")


def test_silu_edges():
    F = 64
    gu = torch.zeros(7, 2 * F, device="cuda").half()
    gu[:, F:] = 1.5
    gu[0, :F] = torch.linspace(-120, 120, F).half()       # beyond the range of exp in fp32
    gu[1, :F] = 65504.0
    gu[2, :F] = -65504.0
    gu[3, 5] = float("nan")
    gu[4, 6] = float("inf")
    gu[5, F + 7] = float("nan")
    ref = silu_ref(gu)
    y = awq.awq_silu_mul(gu)
    rel = 160 * 2.0 ** -23
    check_fp16(y[0:1], ref[0:1], rel, "wide gates")
    assert torch.isinf(y[1]).all() and (y[2] == 0).all() and torch.isnan(y[3, 5]) and torch.isinf(y[4, 6])
    assert torch.isnan(y[5, 7]) and (y[6] == 0).all()
    x8, sx = awq.awq_silu_mul_fp8(gu)
    check_fp8(x8[0:1], sx[0:1], ref[0:1], rel, "wide gates fp8")
    assert sx[1].isfinite() and (x8[1].view(torch.float8_e4m3fn).float() == 448).all()    # 98256 needs no fp16
    assert sx[2] == 0 and (x8[2] == 0).all() and sx[6] == 0 and (x8[6] == 0).all()
    for bad in (3, 4, 5):
        assert not sx[bad].isfinite()


def test_empty_batches_and_given_outputs():
    w = torch.ones(256, device="cuda").half()
    x = torch.empty(0, 256, device="cuda").half()
    assert awq.awq_rmsnorm(x, w, EPS).shape == (0, 256)
    assert awq.awq_silu_mul(x).shape == (0, 128)
    x, r, w = inputs(5, 256)
    y, h = torch.empty_like(x), torch.empty_like(x)
    got = awq.awq_rmsnorm(x, w, EPS, residual=r, h=h, y=y)
    assert got[0] is y and got[1] is h
    with pytest.raises(ValueError):
        awq.awq_rmsnorm(x, w, EPS, y=y[:4])
    with pytest.raises(ValueError):
        awq.awq_rmsnorm(x, w[:128], EPS)
    with pytest.raises(ValueError):
        awq.awq_rmsnorm(x.t().contiguous().t(), w, EPS)
    with pytest.raises(ValueError):
        awq.awq_rmsnorm(x.bfloat16(), w, EPS)
    with pytest.raises(ValueError):
        awq.awq_rmsnorm(x, w, EPS, h=h)
    with pytest.raises(awq.AwqError):
        awq.awq_rmsnorm(x, w, EPS, y=x)
    with pytest.raises(awq.AwqError):
        awq.awq_silu_mul(torch.zeros(2, 24, device="cuda").half())     # F = 12


def test_on_another_stream_and_in_a_graph():
    x, r, w = inputs(64, 4096, seed=9)
    want_y, want_h = awq.awq_rmsnorm(x, w, EPS, residual=r)
    want_s = awq.awq_silu_mul_fp8(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y, h = awq.awq_rmsnorm(x, w, EPS, residual=r)
    s.synchronize()
    assert torch.equal(y, want_y) and torch.equal(h, want_h)
    y, h = torch.zeros_like(y), torch.zeros_like(h)
    x8, sx = torch.zeros_like(want_s[0]), torch.zeros_like(want_s[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        awq.awq_rmsnorm(x, w, EPS, residual=r, h=h, y=y)
        awq.awq_silu_mul_fp8(x, x8=x8, sx=sx)
    for _ in range(3):
        y.zero_(), h.zero_(), x8.zero_(), sx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(h, want_h)
        assert torch.equal(x8, want_s[0]) and torch.equal(sx, want_s[1])


def test_offsets_beyond_32_bits():
    # 2^31 + elements in x and y; the last rows are checked
    K, M = 32768, (1 << 16) + 5
    free, _ = torch.cuda.mem_get_info()
    assert free > 24 << 30
    x = torch.zeros(M, K, dtype=torch.float16, device="cuda")
    tail = slice(M - 4, M)
    g = torch.Generator(device="cuda").manual_seed(8)
    x[tail] = torch.randn(4, K, generator=g, device="cuda").half()
    w = torch.ones(K, device="cuda").half()
    y = awq.awq_rmsnorm(x, w, EPS)
    check_fp16(y[tail], norm_ref(x[tail], w, EPS), fp32_slack(K), "norm")
    del y
    x8, sx = awq.awq_rmsnorm_fp8(x, w, EPS)
    check_fp8(x8[tail], sx[tail], norm_ref(x[tail], w, EPS), fp32_slack(K), "norm fp8")
    del x8
    rel = 32 * 2.0 ** -23
    check_fp16(awq.awq_silu_mul(x)[tail], silu_ref(x[tail]), rel, "silu")
    x8, sx = awq.awq_silu_mul_fp8(x)
    check_fp8(x8[tail], sx[tail], silu_ref(x[tail]), rel, "silu fp8")


@pytest.mark.parametrize("K", [264, 4096, 8192, 20480, 33000])
@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rmsnorm_of_weights_that_are_not_finite(K, with_residual, bad):
    # the formula's y is not finite at that channel (0 * infinity is NaN too), so no row has a finite scale
    x, r, w = inputs(3, K, seed=5)
    x[1], r[1] = 0, 0
    r = r if with_residual else None
    for where in (slice(K // 2, K // 2 + 1), slice(0, K)):
        wb = w.clone()
        wb[where] = bad
        y = awq.awq_rmsnorm(x, wb, EPS, residual=r)
        y = y[0] if with_residual else y
        assert not torch.isfinite(y[:, where]).any(), where
        sx = awq.awq_rmsnorm_fp8(x, wb, EPS, residual=r)[1]
        assert not torch.isfinite(sx).any(), where


# rows beyond 16384 copy the next row ahead while they work: enough rows that
# every CTA walks several
@pytest.mark.parametrize("K", [16392, 20480, 28672, 32768])
@pytest.mark.parametrize("form", ["plain", "residual", "onto x", "onto residual"])
def test_wide_rmsnorm_walks_rows(K, form):
    M = 700
    x, r, w = inputs(M, K, seed=6)
    ref = norm_ref(x, w, EPS, None if form == "plain" else r)
    if form == "plain":
        check_fp16(awq.awq_rmsnorm(x, w, EPS), ref, fp32_slack(K), (form, K))
        check_fp8(*awq.awq_rmsnorm_fp8(x, w, EPS), ref, fp32_slack(K), (form, K))
        return
    want = (x.float() + r.float()).half()
    for fp8 in (False, True):
        xi, ri = x.clone(), r.clone()
        h = {"residual": None, "onto x": xi, "onto residual": ri}[form]
        if fp8:
            x8, sx, h = awq.awq_rmsnorm_fp8(xi, w, EPS, residual=ri, h=h)
            check_fp8(x8, sx, ref, fp32_slack(K), (form, K))
        else:
            y, h = awq.awq_rmsnorm(xi, w, EPS, residual=ri, h=h)
            check_fp16(y, ref, fp32_slack(K), (form, K))
        assert torch.equal(h, want)


@pytest.mark.parametrize("F", [16392, 20480, 28672, 32768])
def test_wide_silu_mul_walks_rows(F):
    g = torch.Generator(device="cuda").manual_seed(F)
    gu = (torch.randn(700, 2 * F, generator=g, device="cuda") * 2).half()
    rel = (float(gu[:, :F].abs().max()) + 16) * 2.0 ** -23
    check_fp8(*awq.awq_silu_mul_fp8(gu), silu_ref(gu), rel, F)
    check_fp16(awq.awq_silu_mul(gu), silu_ref(gu), rel, F)
