"""The dense gated feed-forward block on the GPU: forward, saved projections and gradients, against the formulas
in 64 bits (tests/_llm_ref.py states what the arithmetic may lose)."""
import pytest
import torch

import ternary_rank_weight_b200 as ext
from _llm_ref import ACTS, U, act64, act_eps, act_slope, act_slope2, gated_bound, half_step

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def _make(t, m, n, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 7 * t + 11 * m + 13 * n)
    X = torch.randn(t, n, generator=g, device="cuda").to(dtype)
    Wg = (torch.randn(m, n, generator=g, device="cuda") * n ** -0.5).to(dtype)
    Wu = (torch.randn(m, n, generator=g, device="cuda") * n ** -0.5).to(dtype)
    dH = (0.1 * torch.randn(t, m, generator=g, device="cuda")).to(dtype)
    return X, Wg, Wu, dH


def _proj(X, W):
    """A projection in 64 bits and what n fp32 terms may lose."""
    x, w = X.double(), W.double()
    return x @ w.t(), (W.shape[1] + 24) * U * (x.abs() @ w.abs().t())


def _check_forward(X, Wg, Wu, act, H, G=None, Up=None):
    (g, dg), (u, du) = _proj(X, Wg), _proj(X, Wu)
    h = act64(act, g)[0] * u
    bound = gated_bound(act, g, u, dg, du)
    assert H.dtype == X.dtype and H.shape == h.shape
    assert torch.all((H.double() - h).abs() <= bound * (1 + 2.0 ** -8) + half_step(X.dtype, h))
    if G is not None:
        assert torch.all((G.double() - g).abs() <= dg * (1 + 2.0 ** -8) + half_step(G.dtype, g))
        assert torch.all((Up.double() - u).abs() <= du * (1 + 2.0 ** -8) + half_step(G.dtype, u))


def _check_backward(X, Wg, Wu, dH, act, G, Up, got):
    """The gradients' own arithmetic, from the saved (rounded) projections: dG and dU carry the activation's
    error, two or three fp32 products and one rounding to the operands' type; the sums add theirs."""
    g, u, r, x = G.double(), Up.double(), dH.double(), X.double()
    f, df = act64(act, g)
    # the derivative's parts s, g s, (1 - s) ... carry act_eps each; their magnitudes stay below 1 + slope
    edf = act_eps(g) * (df.abs() + 1 + f.abs()) * 4
    dg, du = r * u * df, r * f
    eg = (r * u).abs() * edf + 4 * U * dg.abs()
    eu = r.abs() * act_eps(g) * f.abs() + 4 * U * du.abs()
    eg = eg + half_step(X.dtype, dg) * (1 + 2.0 ** -8) + eg * 2.0 ** -8
    eu = eu + half_step(X.dtype, du) * (1 + 2.0 ** -8) + eu * 2.0 ** -8
    t, m = g.shape
    wg, wu = Wg.double(), Wu.double()
    dX, dWg, dWu = got
    if dX is not None:
        v = dg @ wg + du @ wu
        e = eg @ wg.abs() + eu @ wu.abs() + (2 * m + 24) * U * ((dg.abs() + eg) @ wg.abs() + (du.abs() + eu) @ wu.abs())
        assert dX.shape == v.shape and torch.all((dX.double() - v).abs() <= e * (1 + 2.0 ** -8) + half_step(X.dtype, v))
    for d, ed, dW in ((dg, eg, dWg), (du, eu, dWu)):
        if dW is not None:
            v = d.t() @ x
            e = ed.t() @ x.abs() + (t + 24) * U * ((d.abs() + ed).t() @ x.abs())
            assert dW.shape == v.shape and torch.all((dW.double() - v).abs() <= e * (1 + 2.0 ** -8) + half_step(X.dtype, v))


SHAPES = [(1, 1, 1), (1, 64, 64), (2, 17, 33), (5, 100, 72), (8, 33, 1000), (9, 40, 64), (16, 130, 777), (17, 16, 16), (31, 129, 200),
          (64, 128, 64), (127, 250, 130), (128, 128, 128), (129, 257, 65), (200, 1000, 300), (300, 1111, 777), (513, 300, 520),
          (1000, 640, 256)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("t,m,n", SHAPES)
def test_forward_matches_64_bits(t, m, n, dtype):
    for act in ACTS:
        X, Wg, Wu, _ = _make(t, m, n, dtype)
        H, G, Up = ext.gated_forward(X, Wg, Wu, act)
        assert G.dtype == Up.dtype == torch.float32
        _check_forward(X, Wg, Wu, act, H, G, Up)
        assert torch.equal(ext.gated(X, Wg, Wu, act), H)
        H2, G2, U2 = ext.gated_forward(X, Wg, Wu, act, save_dtype=dtype)
        assert torch.equal(H2, H) and torch.equal(G2, G.to(dtype)) and torch.equal(U2, Up.to(dtype))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("t,m,n", SHAPES)
def test_backward_matches_64_bits(t, m, n, dtype):
    for act in ACTS:
        X, Wg, Wu, dH = _make(t, m, n, dtype, seed=1)
        for save in (torch.float32, dtype):
            _, G, Up = ext.gated_forward(X, Wg, Wu, act, save_dtype=save)
            got = ext.gated_backward(dH, X, Wg, Wu, G, Up, act)
            _check_backward(X, Wg, Wu, dH, act, G, Up, got)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_small_integers_are_exact(dtype):
    """Integers whose sums stay below 2^8: every product, sum and rounding of the projections and of relu2's
    gradients' sums is exact, so a lost or doubled term anywhere shows."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    t, m, n = 333, 210, 392
    X = (torch.rand(t, n, generator=g, device="cuda") < 0.06).to(dtype)
    Wg = torch.randint(-1, 2, (m, n), generator=g, device="cuda").to(dtype)
    Wu = torch.randint(-1, 2, (m, n), generator=g, device="cuda").to(dtype)
    H, G, Up = ext.gated_forward(X, Wg, Wu, "relu2")
    g64, u64 = X.double() @ Wg.double().t(), X.double() @ Wu.double().t()
    assert g64.abs().max() < 128 and torch.equal(G.double(), g64) and torch.equal(Up.double(), u64)
    assert torch.equal(H, (g64.clamp(min=0) ** 2 * u64).float().to(dtype))
    # gradients with G in {-1, 0, 1}, U in {-1, 0, 1} and sparse dH in {0, 1}: dG, dU small integers
    Gs = torch.randint(-1, 2, (t, m), generator=g, device="cuda").to(dtype)
    Us = torch.randint(-1, 2, (t, m), generator=g, device="cuda").to(dtype)
    dH = (torch.rand(t, m, generator=g, device="cuda") < 0.1).to(dtype)
    dX, dWg, dWu = ext.gated_backward(dH, X, Wg, Wu, Gs, Us, "relu2")
    dg, du = dH.double() * Us.double() * 2 * Gs.double().clamp(min=0), dH.double() * Gs.double().clamp(min=0) ** 2
    for got, want in ((dX, dg @ Wg.double() + du @ Wu.double()), (dWg, dg.t() @ X.double()), (dWu, du.t() @ X.double())):
        assert want.abs().max() < 256 and torch.equal(got.double(), want)


# The shapes of tiles the host picks with 148 SMs: single CTAs 128, 192 and 256 columns wide, pairs 192 and 256 (pairs 128
# wide serve all the small shapes above); the tall ones several tiles a worker.  n is several rings of stages deep, and ragged.
FORWARD_PLANS = [(40, 5501, 453), (17, 9477, 453), (301, 5503, 453), (600, 6903, 453), (301, 6901, 453), (1101, 6905, 453)]
# tokens, m, n, which gradients.  Pairs, dX unsplit, all workers with one dX tile or none, then some with two; single CTAs 256
# wide, dX unsplit and split; dX alone on pairs and on single CTAs; dWg and dWu alone on pairs; split dX and dWg on pairs
BACKWARD_PLANS = [(1101, 6901, 2503, (1, 1, 1)), (2101, 1301, 2507, (1, 1, 1)), (500, 101, 3501, (1, 1, 1)), (3, 5501, 1901, (1, 1, 1)),
                  (901, 101, 2501, (1, 0, 0)), (9, 2003, 2501, (1, 0, 0)), (17, 1001, 131, (0, 1, 1)), (200, 4501, 1003, (1, 1, 0))]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("t,m,n", FORWARD_PLANS)
def test_every_forward_plan(t, m, n, dtype):
    for act, save in (("silu", torch.float32), ("relu2", dtype)):
        X, Wg, Wu, _ = _make(t, m, n, dtype, seed=21)
        H, G, Up = ext.gated_forward(X, Wg, Wu, act, save_dtype=save)
        _check_forward(X, Wg, Wu, act, H, G, Up)
        assert torch.equal(ext.gated(X, Wg, Wu, act), H)
    # whole numbers whose sums are exact (as in test_small_integers_are_exact): a term lost or doubled shows
    X = (X > 1.5).to(dtype)
    Wg, Wu = ((w * n ** 0.5).round().clamp(-1, 1) for w in (Wg, Wu))
    H, G, Up = ext.gated_forward(X, Wg, Wu, "relu2")
    g64, u64 = X.double() @ Wg.double().t(), X.double() @ Wu.double().t()
    assert 16 < g64.abs().max() < 128 and torch.equal(G.double(), g64) and torch.equal(Up.double(), u64)
    assert torch.equal(H, (g64.clamp(min=0) ** 2 * u64).float().to(dtype))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("t,m,n,need", BACKWARD_PLANS)
def test_every_backward_plan(t, m, n, need, dtype):
    X, Wg, Wu, dH = _make(t, m, n, dtype, seed=22)
    _, G, Up = ext.gated_forward(X, Wg, Wu)
    got = ext.gated_backward(dH, X, Wg, Wu, G, Up, need=need)
    assert [v is not None for v in got] == [bool(v) for v in need]
    _check_backward(X, Wg, Wu, dH, "silu", G, Up, got)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(23)
    X = (X > 1.5).to(dtype)
    Wg, Wu = ((w * n ** 0.5).round().clamp(-1, 1) for w in (Wg, Wu))
    G, Up = (torch.randint(-1, 2, (t, m), generator=gen, device="cuda").to(dtype) for _ in range(2))
    dH = (torch.rand(t, m, generator=gen, device="cuda") < 0.1).to(dtype)
    got = ext.gated_backward(dH, X, Wg, Wu, G, Up, "relu2", need=need)
    dg, du = dH.double() * Up.double() * 2 * G.double().clamp(min=0), dH.double() * G.double().clamp(min=0) ** 2
    for a, want in zip(got, (dg @ Wg.double() + du @ Wu.double(), dg.t() @ X.double(), du.t() @ X.double())):
        assert a is None or (want.abs().max() < 256 and want.any() and torch.equal(a.double(), want))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gradients_match_differences_closely(act, dtype):
    """As test_gradients_match_differences, along V = the sign of the exact gradient: every entry then adds its magnitude,
    and the kernels' errors (one rounding of dG or dU, none of G and U, one of the result) stay a small fraction of the
    sum, which is asserted: a gradient of zeros, or of another sign, fails."""
    t, m, n = 40, 96, 72
    X, Wg, Wu, dH = _make(t, m, n, dtype, seed=24)
    _, G, Up = ext.gated_forward(X, Wg, Wu, act)
    grads = ext.gated_backward(dH, X, Wg, Wu, G, Up, act)
    x = [v.double() for v in (X, Wg, Wu)]

    def f(a, b, c):
        return (dH.double() * act64(act, a @ b.t())[0] * (a @ c.t())).sum()

    g, u = x[0] @ x[1].t(), x[0] @ x[2].t()
    a, da = act64(act, g)
    dg, du = dH.double() * u * da, dH.double() * a
    exact = [dg @ x[1] + du @ x[2], dg.t() @ x[0], du.t() @ x[0]]
    terms = [dg.abs() @ x[1].abs() + du.abs() @ x[2].abs(), dg.abs().t() @ x[0].abs(), du.abs().t() @ x[0].abs()]
    # the activation's and its derivative's fp32 errors, as in _check_backward
    ea, eda = act_eps(g) * a.abs(), act_eps(g) * (da.abs() + 1 + a.abs()) * 4
    eg, eu = (dH.double() * u).abs() * eda, dH.double().abs() * ea
    fp32 = [eg @ x[1].abs() + eu @ x[2].abs(), eg.t() @ x[0].abs(), eu.t() @ x[0].abs()]
    half = torch.finfo(dtype).eps / 2
    for i in range(3):
        V = exact[i].sign()
        h = 1e-5
        hi, lo = [v.clone() for v in x], [v.clone() for v in x]
        hi[i] += h * V
        lo[i] -= h * V
        diff = (f(*hi) - f(*lo)) / (2 * h)
        # dG's or dU's rounding in every term, the result's in every entry, sums of 2 m or t terms in fp32; the difference
        # itself is off by the third derivative times (h sum |V W|)^2, below 1e-8, and by 2^-53 / h of the terms
        bound = ((half * 1.01 + (2 * m + 24) * U + 1e-6) * terms[i] + 1.01 * fp32[i] + half * 1.01 * exact[i].abs()).sum()
        assert bound < 0.1 * diff, (bound, diff)
        assert (diff - (grads[i].double() * V).sum()).abs() <= bound


def test_gradients_match_differences():
    """d/ds of sum(dH H(X + s V)) in 64 bits, by central differences of the formula, against the kernels'
    gradients contracted with V: the gradients' bound of one rounding chain (4 roundings of fp16, 2^-11 each,
    of the sum of the terms' magnitudes) and a difference error below 1e-6 of it."""
    t, m, n, act = 40, 96, 72, "gelu"
    X, Wg, Wu, dH = _make(t, m, n, F16, seed=2)
    _, G, Up = ext.gated_forward(X, Wg, Wu, act)
    grads = ext.gated_backward(dH, X, Wg, Wu, G, Up, act)
    x = [X.double(), Wg.double(), Wu.double()]

    def f(a, b, c):
        return (dH.double() * act64(act, a @ b.t())[0] * (a @ c.t())).sum()

    for i in range(3):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(i)
        V = torch.randn(x[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-5
        hi, lo = [v.clone() for v in x], [v.clone() for v in x]
        hi[i] += h * V
        lo[i] -= h * V
        diff = (f(*hi) - f(*lo)) / (2 * h)
        r = dH.double().abs()
        g, u = x[0] @ x[1].t(), x[0] @ x[2].t()
        a, b = r * u.abs() * 1.13, r * 1.13 * g.abs()
        mags = [a @ x[1].abs() + b @ x[2].abs(), a.t() @ x[0].abs(), b.t() @ x[0].abs()][i]
        # G and U rounded once each and act', act of a rounded G (slopes 0.8 and 1.13 of 2^-11 |G|), dG, the result
        bound = 8 * 2.0 ** -11 * (mags * (1 + g.abs().max()) * V.abs()).sum()
        assert (diff - (grads[i].double() * V).sum()).abs() <= bound


def test_large_magnitudes_of_the_gate():
    """Gates far out on both sides: silu and its gradient reach their limits without NaN."""
    n = 64
    X = torch.eye(n, device="cuda", dtype=BF16)
    vals = torch.tensor([-3e38, -1e30, -200.0, -90.0, -88.0, -20.0, -1.0, 0.0, 1.0, 20.0, 88.0, 90.0, 200.0, 1e18], device="cuda")
    Wg = torch.zeros(n, n, device="cuda")
    Wg[:, :14] = vals
    Wg, Wu = Wg.to(BF16), torch.ones(n, n, device="cuda").to(BF16)
    for act in ("silu", "gelu", "gelu_tanh"):
        H, G, Up = ext.gated_forward(X, Wg, Wu, act)
        want = act64(act, Wg.double().t())[0].to(torch.float32).to(BF16)
        assert torch.isfinite(H).all()
        assert torch.all((H.double() - want.double()).abs() <= 2.0 ** -7 * want.double().abs() + 1e-9)
        for g in ext.gated_backward(torch.ones_like(H), X, Wg, Wu, G, Up, act):
            assert not torch.isnan(g).any()


def test_relu2_of_an_overflowed_gate():
    """A projection past the 16-bit range: relu2 and its gradient are 0 on the negative side."""
    X = torch.full((1, 64), 60000.0, dtype=F16, device="cuda")
    Wg, Wu = torch.full((16, 64), -60000.0, dtype=F16, device="cuda"), torch.ones(16, 64, dtype=F16, device="cuda")
    for t in (1, 20):
        H, G, Up = ext.gated_forward(X.expand(t, 64), Wg, Wu * 1e-4, "relu2", save_dtype=F16)
        assert not H.any() and torch.isinf(G).all()
        for g in ext.gated_backward(torch.ones_like(H), X.expand(t, 64), Wg, Wu * 1e-4, G, Up, "relu2"):
            assert not g.any()


@pytest.mark.parametrize("act", ACTS)
def test_a_gate_below_the_fp32_range(act):
    """Sums past -3.4e38 are -inf in fp32: every activation is 0 there (and inf above, where U is not 0)."""
    for t in (1, 20):
        X = torch.full((t, 64), 2.0 ** 70, dtype=BF16, device="cuda")
        Wg = torch.full((24, 64), -2.0 ** 70, dtype=BF16, device="cuda")
        Wg[1::2] *= -1
        Wu = torch.full((24, 64), 2.0 ** -70, dtype=BF16, device="cuda")
        H, G, Up = ext.gated_forward(X, Wg, Wu, act)
        assert torch.isinf(G).all() and not H[:, ::2].any() and torch.isposinf(H[:, 1::2]).all()
        Wg[2, 5] = float("nan")
        assert torch.isnan(ext.gated(X, Wg, Wu, act)[:, 2]).all()
        for dtype in (torch.float32, BF16):              # 4-bit weights: -7 s and 7 s of the greatest scale, X in the range
            W = torch.full((24, 64), -4.4e5, device="cuda")
            W[1::2] *= -1
            w, one = ext.int4_quantize(W, 64, affine=False), ext.int4_quantize(torch.ones(24, 64, device="cuda"), 64, affine=False)
            for rows in (1, 20):
                Z = torch.full((rows, 64), 2.0 ** 114, dtype=dtype, device="cuda")
                h = ext.int4_gated(w, one, Z, act)
                assert not h[:, ::2].any() and torch.isposinf(h[:, 1::2]).all()


@pytest.mark.parametrize("dtype,save", [(F16, F16), (F16, torch.float32), (BF16, BF16), (BF16, torch.float32)])
@pytest.mark.parametrize("act", ACTS)
def test_gradients_of_infinite_projections(act, dtype, save):
    """Saved projections that are infinite count as the type's largest value: act is then 0 or g (relu2 0 or g^2), act'
    0 or 1 (relu2 0 or 2 g), and nothing becomes NaN.  Where the products leave the range, dH is 0 and so are they."""
    inf, big = float("inf"), torch.finfo(save).max
    for t in (1, 20):
        m, n = 24, 40
        X, Wg, Wu, _ = _make(t, m, n, dtype, seed=9)
        gv = torch.tensor([inf, -inf, inf, -inf, 1.0, 1.0] * 4, dtype=torch.float64, device="cuda")
        uv = torch.tensor([0.5, 0.5, inf, -inf, inf, 0.5] * 4, dtype=torch.float64, device="cuda")
        dH = torch.full((t, m), 2.0 ** -22, dtype=dtype, device="cuda")
        if save != F16:                                 # past every 16-bit product: gradients of 0
            dH[:, (gv > 0) & (torch.isinf(gv) | torch.isinf(uv))] = 0
        elif act == "relu2":
            dH[:, 2::6] = 0                             # 2 65504^2 of it
        G, Up = gv.to(save).expand(t, m).contiguous(), uv.to(save).expand(t, m).contiguous()
        g, u = gv.clamp(-big, big), uv.clamp(-big, big)
        f, df = act64(act, torch.where(g.abs() > 1, g.sign(), g))
        far = g.abs() > 1
        pos = (g > 0).double()
        f = torch.where(far, pos * (g * g if act == "relu2" else g), f)
        df = torch.where(far, pos * (2 * g if act == "relu2" else 1.0), df)
        r = dH.double()
        dg, du = r * df * u, r * f
        assert max(dg.abs().max(), du.abs().max()) < (65000 if dtype == F16 else 3e38)
        # the limits are exact, the activation at 1 has its error (as in _check_backward); products and one rounding
        edf, ef = (torch.where(far, 0.0, act_eps(g) * v) for v in ((df.abs() + 1 + f.abs()) * 4, f.abs()))
        eg, eu = (r * u).abs() * edf + 4 * U * dg.abs(), r.abs() * ef + 4 * U * du.abs()
        eg, eu = (e * (1 + 2.0 ** -8) + half_step(dtype, v) * (1 + 2.0 ** -8) for e, v in ((eg, dg), (eu, du)))
        got = ext.gated_backward(dH, X, Wg, Wu, G, Up, act)
        x, wg, wu = X.double(), Wg.double(), Wu.double()
        want = (dg @ wg + du @ wu, dg.t() @ x, du.t() @ x)
        err = (eg @ wg.abs() + eu @ wu.abs(), eg.t() @ x.abs(), eu.t() @ x.abs())
        mag = (dg.abs() @ wg.abs() + du.abs() @ wu.abs(), dg.abs().t() @ x.abs(), du.abs().t() @ x.abs())
        for a, v, e, s in zip(got, want, err, mag):
            assert torch.all((a.double() - v).abs() <= (e + (2 * m + 24) * U * (s + e)) * (1 + 2.0 ** -8) + half_step(dtype, v))
        G[-1, 3] = float("nan")                         # NaN is passed on
        dX, dWg, dWu = ext.gated_backward(dH, X, Wg, Wu, G, Up, act)
        assert torch.isnan(dX[-1]).all() and torch.isnan(dWg[3]).all() and torch.isnan(dWu[3]).all()
        keep = [i for i in range(m) if i != 3]
        assert not torch.isnan(dX[:-1]).any() and torch.equal(dWg[keep], got[1][keep]) and torch.equal(dWu[keep], got[2][keep])


# tokens, m, n: single CTAs; pairs; a split dX on pairs; several tiles a worker, pairs
@pytest.mark.parametrize("t,m,n", [(20, 100, 72), (300, 1111, 777), (130, 4095, 1000), (1100, 6900, 500)])
def test_waits_that_run_out_end_with_a_status(t, m, n):
    """The products of one worker are withheld (a host-set flag): every wait for them gives up, the status says so, and
    the next call is as ever."""
    X, Wg, Wu, dH = _make(t, m, n, BF16, seed=11)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = ext.gated_forward(X, Wg, Wu, async_status=st)
    gref = ext.gated_backward(dH, X, Wg, Wu, *ref[1:], async_status=st)
    assert int(st.item()) == 0
    for worker in (1, 2):
        with ext.debug_wait_fault(worker):
            ext.gated_forward(X, Wg, Wu, async_status=st)
            late = int(st.item())
            ext.gated_backward(dH, X, Wg, Wu, *ref[1:], async_status=st)
        assert late == ext.STATUS["ETIMEOUT"] and int(st.item()) == ext.STATUS["ETIMEOUT"]
        again = ext.gated_forward(X, Wg, Wu, async_status=st)
        assert int(st.item()) == 0 and all(torch.equal(a, b) for a, b in zip(again, ref))
        again = ext.gated_backward(dH, X, Wg, Wu, *ref[1:], async_status=st)
        assert int(st.item()) == 0 and all(torch.equal(a, b) for a, b in zip(again, gref))


@pytest.mark.parametrize("save", [torch.float32, BF16])
@pytest.mark.parametrize("t,m,n", [(20, 100, 72), (300, 1111, 777), (130, 4095, 1000), (1100, 6900, 500)])
def test_waits_that_run_out_leave_nan(t, m, n, save):
    """Without a status the outputs themselves show it: what the withheld worker did not reach is NaN, all else is right."""
    X, Wg, Wu, dH = _make(t, m, n, BF16, seed=12)
    ref = ext.gated_forward(X, Wg, Wu, save_dtype=save)
    gref = ext.gated_backward(dH, X, Wg, Wu, *ref[1:])
    torch.full((8, *gref[1].shape), 7.0, device="cuda")              # memory that the next outputs may get
    with ext.debug_wait_fault(1):
        got = ext.gated_forward(X, Wg, Wu, save_dtype=save)
        ggot = ext.gated_backward(dH, X, Wg, Wu, *ref[1:])
        alone = ext.gated_backward(dH, X, Wg, Wu, *ref[1:], need=(False, True, True))
    nan = [torch.isnan(v) for v in got]
    assert nan[0].any() and not nan[0].all() and torch.equal(nan[0], nan[1]) and torch.equal(nan[0], nan[2])
    assert any(torch.isnan(v).any() for v in ggot) and any(torch.isnan(v).any() for v in alone[1:])
    for a, b in zip((*got, *ggot, *alone[1:]), (*ref, *gref, *gref[1:])):
        assert torch.equal(torch.where(torch.isnan(a), b, a), b)


def test_shapes_strides_and_partial_gradients():
    t, m, n = 60, 130, 100
    X, Wg, Wu, dH = _make(t, m, n, BF16)
    H, G, Up = ext.gated_forward(X, Wg, Wu)
    for lead in ((3, 20), (2, 5, 6)):
        H2, G2, U2 = ext.gated_forward(X.view(*lead, n), Wg, Wu)
        assert H2.shape == (*lead, m) and torch.equal(H2.view(t, m), H) and torch.equal(G2.view(t, m), G)
        dX, dWg, dWu = ext.gated_backward(dH.view(*lead, m), X.view(*lead, n), Wg, Wu, G2, U2)
        assert dX.shape == (*lead, n)
    ref = ext.gated_backward(dH, X, Wg, Wu, G, Up)
    assert torch.equal(dX.view(t, n), ref[0]) and torch.equal(dWg, ref[1]) and torch.equal(dWu, ref[2])
    for need in ((True, False, False), (False, True, False), (False, False, True), (True, False, True), (False, False, False)):
        got = ext.gated_backward(dH, X, Wg, Wu, G, Up, need=need)
        for want, a, b in zip(need, got, ref):
            assert (a is None) == (not want) and (a is None or torch.equal(a, b))
    one = ext.gated(X[0], Wg, Wu)
    assert one.shape == (m,) and torch.equal(one, ext.gated(X[:1], Wg, Wu)[0])
    # rows off the 16-byte boundaries, strided rows, transposed storage
    bigX, bigW, bigd = torch.zeros(t, n + 9, dtype=BF16, device="cuda"), torch.zeros(m, n + 16, dtype=BF16, device="cuda"), \
        torch.zeros(t, m + 3, dtype=BF16, device="cuda")
    bigX[:, 5:5 + n], bigW[:, 8:8 + n], bigd[:, 1:1 + m] = X, Wg, dH
    Xv, Wv, dv, Wt = bigX[:, 5:5 + n], bigW[:, 8:8 + n], bigd[:, 1:1 + m], Wu.t().contiguous().t()
    H3, G3, U3 = ext.gated_forward(Xv, Wv, Wt)
    assert torch.equal(H3, H) and torch.equal(G3, G) and torch.equal(U3, Up)
    for a, b in zip(ext.gated_backward(dv, Xv, Wv, Wt, G3.new_zeros(t, m + 3)[:, :m].copy_(G3), U3), ref):
        assert torch.equal(a, b)
    out = torch.full((t + 2, m + 7), 5.0, dtype=BF16, device="cuda")
    got = ext.gated(X, Wg, Wu, out=out[1:-1, 3:3 + m])
    assert torch.equal(got, H)
    out[1:-1, 3:3 + m] = 5.0
    assert torch.all(out == 5.0)


@pytest.mark.parametrize("t,m,n", [(40, 2100, 300), (100, 2560, 128), (200, 3000, 40), (130, 4095, 1000)])
def test_split_depth_of_few_tokens(t, m, n):
    """With few tokens the 2 m terms of dX are summed in shares."""
    X, Wg, Wu, dH = _make(t, m, n, BF16, seed=4)
    _, G, Up = ext.gated_forward(X, Wg, Wu, "gelu")
    got = ext.gated_backward(dH, X, Wg, Wu, G, Up, "gelu")
    _check_backward(X, Wg, Wu, dH, "gelu", G, Up, got)
    again = ext.gated_backward(dH, X, Wg, Wu, G, Up, "gelu", need=(True, False, False))
    assert torch.equal(again[0], got[0])


def test_outputs_that_share_memory_with_inputs_are_refused():
    """In place, a row's results would be written while other CTAs still read the row."""
    X, Wg, Wu, _ = _make(40, 64, 64, BF16, seed=14)
    w = ext.int4_quantize(Wg, 64)
    ref, y, h = ext.gated(X, Wg, Wu), ext.int4_matvec(w, X), ext.int4_gated(w, w, X)
    for call in (lambda o: ext.gated(X, Wg, Wu, out=o), lambda o: ext.int4_matvec(w, X, out=o), lambda o: ext.int4_gated(w, w, X, out=o)):
        with pytest.raises(ValueError, match="share memory"):
            call(X)
    with pytest.raises(ValueError, match="share memory"):
        ext.gated(X, Wg, Wu, out=Wg[:40])
    # side by side in one buffer is fine
    both = torch.zeros(40, 128, dtype=BF16, device="cuda")
    both[:, :64] = X
    for call, want in ((lambda x, o: ext.gated(x, Wg, Wu, out=o), ref), (lambda x, o: ext.int4_matvec(w, x, out=o), y),
                       (lambda x, o: ext.int4_gated(w, w, x, out=o), h)):
        call(both[:, :64], both[:, 64:])
        assert torch.equal(both[:, 64:], want) and torch.equal(both[:, :64], X)


def test_one_vector_and_broadcast_gradient():
    X, Wg, Wu, _ = _make(1, 70, 40, BF16, seed=5)
    H, G, Up = ext.gated_forward(X[0], Wg, Wu)
    assert H.shape == G.shape == (70,)
    dH = torch.ones(1, dtype=BF16, device="cuda").expand(70)
    dX, dWg, dWu = ext.gated_backward(dH, X[0], Wg, Wu, G, Up)
    assert dX.shape == (40,)
    _check_backward(X, Wg, Wu, dH.contiguous()[None], "silu", G[None], Up[None], (dX[None], dWg, dWu))


def test_calls_on_two_streams_at_once():
    a, b = _make(300, 700, 400, BF16, seed=6), _make(20, 900, 640, BF16, seed=7)
    refs = [ext.gated_forward(*v[:3]) for v in (a, b)]
    grads = [ext.gated_backward(v[3], *v[:3], *r[1:]) for v, r in zip((a, b), refs)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(10):
        for i, v in enumerate((a, b)):
            f = ext.gated_forward(*v[:3], stream=s[i])
            outs.append((i, f, ext.gated_backward(v[3], *v[:3], *f[1:], stream=s[i])))
    torch.cuda.synchronize()
    for i, f, g in outs:
        assert all(torch.equal(p, q) for p, q in zip((*f, *g), (*refs[i], *grads[i])))


def test_host_threads_at_once():
    """Several host threads, each on a stream of its own, through every kernel whose launch keeps something per device."""
    from concurrent.futures import ThreadPoolExecutor
    X, Wg, Wu, dH = _make(200, 256, 384, F16, seed=13)
    w = ext.int4_quantize(Wg, 64)

    def calls(stream):
        f = ext.gated_forward(X, Wg, Wu, stream=stream)
        return (*f, *ext.gated_backward(dH, X, Wg, Wu, *f[1:], stream=stream), ext.int4_matvec(w, X[:3], stream=stream),
                ext.int4_matvec(w, X[:30], stream=stream), ext.int4_gated(w, w, X[:64], stream=stream))

    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(8)]
    with ThreadPoolExecutor(8) as pool:
        got = list(pool.map(calls, streams))
    torch.cuda.synchronize()
    ref = calls(None)
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, ref))


def test_results_past_32_bit_offsets():
    """2.4 G entries of H: the last tokens' are those of a call of their own."""
    t, m, n = 40100, 60000, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    X = torch.randn(t, n, generator=g, device="cuda").to(BF16)
    Wg, Wu = (torch.randn(m, n, generator=g, device="cuda").to(BF16) * 0.125 for _ in range(2))
    H = ext.gated(X, Wg, Wu)
    assert torch.equal(H[-100:], ext.gated(X[-100:], Wg, Wu)) and torch.equal(H[:100], ext.gated(X[:100], Wg, Wu))


def test_no_tokens():
    X, Wg, Wu, dH = _make(4, 40, 24, F16)
    H, G, Up = ext.gated_forward(X[:0], Wg, Wu)
    assert H.shape == (0, 40) and G.shape == (0, 40)
    dX, dWg, dWu = ext.gated_backward(dH[:0], X[:0], Wg, Wu, G, Up)
    assert dX.shape == (0, 24) and not dWg.any() and not dWu.any() and dWg.shape == (40, 24)


def test_nan_stays_in_its_token():
    X, Wg, Wu, dH = _make(140, 70, 200, BF16)
    ref = ext.gated(X, Wg, Wu)
    X[3, 5] = float("nan")
    got = ext.gated(X, Wg, Wu)
    keep = [i for i in range(140) if i != 3]
    assert torch.equal(got[keep], ref[keep]) and torch.isnan(got[3]).all()


def test_columns_beside_the_inputs_are_not_read():
    """Padding columns and neighbouring rows hold NaN; none of it may enter a sum."""
    for t in (3, 150):
        X, Wg, Wu, dH = _make(t, 75, 100, BF16)
        ref = ext.gated_forward(X, Wg, Wu)
        gref = ext.gated_backward(dH, X, Wg, Wu, *ref[1:])

        def surround(a):
            b = torch.full((a.shape[0] + 8, a.shape[1] + 20), float("nan"), dtype=a.dtype, device="cuda")
            b = b[:, :b.shape[1] // 8 * 8].contiguous()
            v = b[4:4 + a.shape[0], 8:8 + a.shape[1]]
            v.copy_(a)
            return v

        Xs, Gs, Us = surround(X), surround(Wg), surround(Wu)
        got = ext.gated_forward(Xs, Gs, Us)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        got = ext.gated_backward(surround(dH), Xs, Gs, Us, surround(ref[1]), surround(ref[2]))
        assert all(torch.equal(a, b) for a, b in zip(got, gref))


def test_repeats_bit_for_bit_on_streams_and_in_graphs():
    for t in (5, 300):
        X, Wg, Wu, dH = _make(t, 520, 260, BF16)
        fw = ext.gated_forward(X, Wg, Wu, "gelu_tanh")
        ref = (*fw, *ext.gated_backward(dH, X, Wg, Wu, fw[1], fw[2], "gelu_tanh"))
        torch.cuda.synchronize()
        st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
        s = torch.cuda.Stream()
        for _ in range(3):
            a = ext.gated_forward(X, Wg, Wu, "gelu_tanh", stream=s, async_status=st)
            b = ext.gated_backward(dH, X, Wg, Wu, a[1], a[2], "gelu_tanh", stream=s.cuda_stream)
            s.synchronize()
            assert all(torch.equal(p, q) for p, q in zip((*a, *b), ref)) and int(st.item()) == 0
        graphs = []
        for _ in range(2):                      # two graphs alive at once
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                a = ext.gated_forward(X, Wg, Wu, "gelu_tanh")
                b = ext.gated_backward(dH, X, Wg, Wu, a[1], a[2], "gelu_tanh", async_status=st)
            graphs.append((gr, (*a, *b)))
        for gr, outs in graphs + graphs:
            for o in outs:
                o.zero_()
            gr.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(outs, ref)) and int(st.item()) == 0


def test_block_in_4_bits_follows_the_dense_block():
    """A converted MLP as it is used: quantise gate, up and down, run tokens through the 4-bit block and the
    4-bit down projection, and through the dense block over the values the 4 bits stand for (rounded to
    fp16, 2^-11 of each weight)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    m, n = 700, 256
    Wg, Wu, Wd = (torch.randn(*s, generator=g, device="cuda") * s[1] ** -0.5 for s in ((m, n), (m, n), (n, m)))
    wg, wu, wd = (ext.int4_quantize(w, 64) for w in (Wg, Wu, Wd))
    dg, du, dd = (ext.int4_dequantize(w, F16) for w in (wg, wu, wd))
    for t in (1, 12, 90):
        X = torch.randn(t, n, generator=g, device="cuda").to(F16)
        h4 = ext.int4_gated(wg, wu, X)
        y4 = ext.int4_matvec(wd, h4)
        h16 = ext.gated(X, dg, du)
        x = X.double()
        G, Up = x @ dg.double().t(), x @ du.double().t()
        eg, eu = (2.0 ** -10 * (x.abs() @ w.double().abs().t()) for w in (dg, du))
        bound = gated_bound("silu", G, Up, eg, eu)
        assert torch.all((h4.double() - h16.double()).abs() <= 2 * bound + 3 * half_step(F16, h16.double()))
        y = h4.double() @ ext.int4_dequantize(wd).double().t()
        mag = h4.double().abs() @ (dd.double().abs() + 2 * wd.scale.double().max() * 8).t()
        assert torch.all((y4.double() - y).abs() <= (64 + 2 * 11 + 20) * U * 4 * mag + half_step(F16, y))


def test_library_refuses_bad_arguments():
    L, einval = ext._lib.load(), ext.STATUS["EINVAL"]
    t, m, n = 20, 24, 32
    X, Wg, Wu, dH = _make(t, m, n, BF16)
    H, G, Up = ext.gated_forward(X, Wg, Wu)
    out = [torch.zeros(s, dtype=BF16, device="cuda") for s in ((t, n), (m, n), (m, n))]
    need = L.externd_gated_backward_work(m, n, t)
    work = torch.zeros(need + 3 * L.externd_aligned_bytes(2, m, n), dtype=torch.uint8, device="cuda")
    host = torch.zeros(1 << 16, dtype=torch.uint8)
    st = torch.cuda.current_stream().cuda_stream
    base = dict(x=X.data_ptr(), ldx=n, wg=Wg.data_ptr(), ldg=n, wu=Wu.data_ptr(), ldu=n, dt=2, m=m, n=n, t=t, act=0, h=H.data_ptr(),
                ldh=m, g=G.data_ptr(), u=Up.data_ptr(), ldgu=m, sd=0, fw=None, fwb=0, status=None, dh=dH.data_ptr(), lddh=m, dx=out[0].data_ptr(), lddx=n,
                dwg=out[1].data_ptr(), dwu=out[2].data_ptr(), lddw=n, work=work.data_ptr(), wb=need)

    def fwd(**kw):
        a = dict(base, **kw)
        return L.externd_gated(*(a[k] for k in "x ldx wg ldg wu ldu dt m n t act h ldh g u sd ldgu fw fwb status".split()), st)

    def bwd(**kw):
        a = dict(base, **kw)
        return L.externd_gated_backward(*(a[k] for k in "dh lddh x ldx wg ldg wu ldu g u sd ldgu dt m n t act dx lddx dwg dwu lddw work "
                                          "wb status".split()), st)

    assert fwd() == 0 and bwd() == 0 and fwd(g=None, u=None) == 0
    common = [dict(x=None), dict(wg=None), dict(wu=None), dict(dt=0), dict(dt=5), dict(m=0), dict(n=0), dict(t=-1), dict(act=4),
              dict(act=-1), dict(ldx=n + 1), dict(ldx=n - 8), dict(ldg=n + 4), dict(ldu=n - 8), dict(x=X.data_ptr() + 2),
              dict(wg=Wg.data_ptr() + 1), dict(wg=Wg.data_ptr() + 8), dict(sd=1), dict(sd=7), dict(x=host.data_ptr()), dict(wu=host.data_ptr()), dict(status=host.data_ptr()),
              dict(u=None), dict(ldgu=m - 1), dict(g=G.data_ptr() + 1)]
    for kw in common:
        assert fwd(**kw) == einval, kw
        assert bwd(**kw) == einval, kw
    for kw in (dict(h=None), dict(ldh=m - 1), dict(h=host.data_ptr()), dict(g=None)):
        assert fwd(**kw) == einval, kw
    for kw in (dict(dh=None), dict(lddh=m - 1), dict(dx=host.data_ptr()), dict(lddx=n - 1), dict(lddw=n - 1), dict(work=None),
               dict(wb=need - 1), dict(work=work.data_ptr() + 16), dict(dwg=host.data_ptr())):
        assert bwd(**kw) == einval, kw
    # rows off the 16-byte boundaries take their place in work
    over = (work.data_ptr(), L.externd_aligned_bytes(2, t, n))
    assert fwd(x=X.data_ptr() + 2, t=t - 1, fw=over[0], fwb=over[1]) == 0
    assert fwd(x=X.data_ptr() + 2, t=t - 1, fw=over[0], fwb=L.externd_aligned_bytes(2, t - 1, n) - 1) == einval
    assert bwd(x=X.data_ptr() + 2, t=t - 1, wb=need + over[1]) == 0
    assert bwd(dx=None, wg=None, wu=None) == 0 and bwd(dwg=None, dwu=None, x=None) == 0
    with pytest.raises(ValueError):
        ext.gated(X.float(), Wg.float(), Wu.float())
    with pytest.raises(ValueError):
        ext.gated(X, Wg, Wu.half())
    with pytest.raises(ValueError):
        ext.gated(X, Wg, Wu[:-1])
    with pytest.raises(ValueError):
        ext.gated_backward(dH[:-1], X, Wg, Wu, G, Up)
