"""4-bit weights with group scales on the GPU: quantiser, values, products and the gated form, against plain
64-bit forms (tests/_llm_ref.py states what the arithmetic may lose)."""
import numpy as np
import pytest
import torch

import ternary_rank_weight_b200 as ext
from _llm_ref import ACTS, U, act64, gated_bound, half_step, quantize64

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _matrix(m, n, seed, dtype=F32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randn(m, n, generator=g, device="cuda") * 0.02
    return (w * torch.exp(0.5 * torch.randn(m, 1, generator=g, device="cuda"))).to(dtype)


def _vectors(t, n, seed, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 + seed)
    return torch.randn(t, n, generator=g, device="cuda").to(dtype)


def _random_weights(m, n, group, affine, seed):
    """Any codes (the padding columns' too), scales and offsets, also ones no quantiser would choose."""
    rng = np.random.default_rng(seed)
    q = torch.from_numpy(rng.integers(0, 256, size=(m, ext.int4_row_bytes(n)), dtype=np.uint8)).cuda()
    groups = (n + group - 1) // group
    s = torch.from_numpy((0.01 * np.exp(rng.standard_normal((groups, m)))).astype(np.float16)).cuda()
    b = torch.from_numpy((0.01 * rng.standard_normal((groups, m))).astype(np.float16)).cuda() if affine else None
    return ext.Int4Weights(q, s, b, m, n, group)


def _values64(w):
    """The matrix and the magnitudes of its two parts, in 64 bits, from the documented layout."""
    q = torch.from_numpy(w.codes()).cuda().double() - 8
    s = w.scale.double().t().repeat_interleave(w.group, 1)[:, :w.n]
    b = torch.zeros_like(q) if w.offset is None else w.offset.double().t().repeat_interleave(w.group, 1)[:, :w.n]
    return s * q + b, (s * q).abs() + b.abs()


def _sum_bound(w, mag, x):
    """A group's sum has group terms (three parts each for fp32 vectors); the groups' sums, scaled, meet in
    at most 2 ceil(n / group) + 20 more additions."""
    parts = 3 if x.dtype == F32 else 1
    return (parts * w.group + 2 * ((w.n + w.group - 1) // w.group) + 20) * U * (x.double().abs() @ mag.t())


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("m,n,group", [(1, 1, 32), (3, 31, 32), (5, 129, 32), (17, 128, 64), (7, 300, 64), (33, 1000, 128),
                                       (300, 257, 128), (64, 2048, 128)])
def test_quantize_matches_the_definition_exactly(m, n, group, affine, dtype):
    A = _matrix(m, n, m + n, dtype)
    w = ext.int4_quantize(A, group, affine=affine)
    codes, scale, offset, values = quantize64(A, group, affine)
    assert torch.equal(w.scale, scale)
    assert (w.offset is None) == (not affine)
    if affine:
        assert torch.equal(w.offset, offset)
    got = torch.from_numpy(w.codes()).cuda()
    assert torch.equal(got, codes)
    full = ext.unpack_int4(w.q.cpu().numpy(), ext.int4_row_bytes(n) * 2)
    assert np.all(full[:, n:] == 8)
    for out in (F32, F16, BF16):
        v = ext.int4_dequantize(w, out).double()
        assert torch.all((v - values).abs() <= half_step(out, values))


def test_quantize_decides_ties_as_64_bits_do():
    """Entries on and within one fp32 step of every border between codes."""
    s = 0.5                                            # symmetric: max |A| = 3.5 gives s = 0.5 exactly
    mids = torch.arange(-7, 7, dtype=torch.float64) * s + s / 2
    rows = []
    for d in (-1, 0, 1):
        row = torch.zeros(32, dtype=torch.float32)
        row[:14] = mids.float()
        row[:14] = torch.where(torch.tensor(d == 0), row[:14],
                               torch.nextafter(row[:14], torch.full((14,), float("inf") if d > 0 else -float("inf"))))
        row[20] = 3.5
        rows.append(row)
    for scale in (1.0, 1 / 3, 1e-3, 7e-5, 1e-6, 1e4):
        A = (torch.stack(rows) * scale).cuda()
        for affine in (False, True):
            w = ext.int4_quantize(A, 32, affine=affine)
            codes, sc, off, _ = quantize64(A, 32, affine)
            assert torch.equal(w.scale, sc) and (not affine or torch.equal(w.offset, off))
            assert torch.equal(torch.from_numpy(w.codes()).cuda(), codes), (scale, affine)


def test_quantize_constant_zero_and_tiny_groups():
    A = torch.zeros(4, 96, device="cuda")
    A[1] = 0.37
    A[2] = -1e-9                                        # below the fp16 scales: the scale is 0
    A[3, :32] = torch.linspace(-1e-7, 1e-7, 32)
    for affine in (False, True):
        w = ext.int4_quantize(A, 32, affine=affine)
        codes, sc, off, values = quantize64(A, 32, affine)
        assert torch.equal(w.scale, sc) and torch.equal(torch.from_numpy(w.codes()).cuda(), codes)
        assert torch.equal(ext.int4_dequantize(w).double(), values.float().double())


@pytest.mark.parametrize("bad,status", [(float("nan"), "ENONFINITE"), (float("inf"), "ENONFINITE"),
                                        (-float("inf"), "ENONFINITE"), (1e7, "ELIMIT"), (3e38, "ELIMIT")])
def test_quantize_reports_values_it_cannot_hold(bad, status):
    A = _matrix(9, 200, 1)
    A[4, 130] = bad
    with pytest.raises(ext.ExterndError) as e:
        ext.int4_quantize(A, 64)
    assert e.value.status == ext.STATUS[status]
    st = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    w = ext.int4_quantize(A, 64, async_status=st)
    assert int(st.item()) == ext.STATUS[status]
    good = quantize64(A[:4], 64, True)                 # the other rows are as ever
    assert torch.equal(torch.from_numpy(w.codes()[:4]).cuda(), good[0])
    A[4, 130] = 1.0
    ext.int4_quantize(A, 64, async_status=st)
    assert int(st.item()) == 0
    B = _matrix(9, 200, 1)                             # NaN is reported before a range error
    B[0, 0], B[5, 150] = 1e7, float("nan")
    ext.int4_quantize(B, 64, async_status=st)
    assert int(st.item()) == ext.STATUS["ENONFINITE"]


def test_quantize_takes_strided_rows():
    big = _matrix(40, 333, 5)
    for view in (big[:, 1:200], big[::2, 3:], big.t()):
        w = ext.int4_quantize(view, 64)
        ref = ext.int4_quantize(view.contiguous(), 64)
        assert torch.equal(w.q, ref.q) and torch.equal(w.scale, ref.scale) and torch.equal(w.offset, ref.offset)


MATVEC = [(1, 1, 1, 32), (1, 16, 128, 128), (2, 17, 129, 64), (3, 33, 31, 32), (8, 100, 777, 64), (9, 40, 256, 128),
          (1, 300, 2560, 128), (31, 65, 500, 32), (33, 50, 1000, 64), (64, 130, 384, 128), (65, 16, 200, 32),
          (130, 200, 1024, 128), (300, 31, 300, 64)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("t,m,n,group", MATVEC)
def test_matvec_matches_64_bits(t, m, n, group, affine, dtype):
    w = _random_weights(m, n, group, affine, seed=t + m + n)
    X = _vectors(t, n, t, dtype)
    W, mag = _values64(w)
    y = X.double() @ W.t()
    got = ext.int4_matvec(w, X)
    assert got.dtype == dtype and got.shape == (t, m)
    assert torch.all((got.double() - y).abs() <= _sum_bound(w, mag, X) * (1 + 2.0 ** -8) + half_step(dtype, y))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("t", [1, 5, 16, 40, 64, 100])
def test_matvec_small_integers_are_exact(t, dtype):
    """Integer vectors, scales that are powers of two, integer offsets: every sum is an integer (in units of
    1/2) far below 2^24, so nothing may be lost before the last rounding."""
    rng = np.random.default_rng(t)
    m, n, group = 75, 450, 64
    w = _random_weights(m, n, group, True, seed=t)
    w.scale.copy_(torch.from_numpy(rng.choice([0.5, 1.0, 2.0], size=tuple(w.scale.shape)).astype(np.float16)))
    w.offset.copy_(torch.from_numpy(rng.integers(-3, 4, size=tuple(w.scale.shape)).astype(np.float16)))
    X = torch.from_numpy(rng.integers(-8, 9, size=(t, n))).cuda().to(dtype)
    y = X.double() @ _values64(w)[0].t()
    assert torch.equal(ext.int4_matvec(w, X), y.float().to(dtype))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t,m,n,group", [(1, 1, 1, 32), (1, 100, 640, 128), (3, 33, 200, 64), (8, 48, 777, 32), (17, 50, 300, 64),
                                         (40, 130, 512, 128), (100, 20, 260, 32)])
def test_gated_matches_64_bits(t, m, n, group, act, dtype):
    wg, wu = _random_weights(m, n, group, t % 2 == 1, seed=t), _random_weights(m, n, group, True, seed=t + 1)
    X = _vectors(t, n, t, dtype) * 0.5
    (Wg, mg), (Wu, mu) = _values64(wg), _values64(wu)
    g, u = X.double() @ Wg.t(), X.double() @ Wu.t()
    h = act64(act, g)[0] * u
    got = ext.int4_gated(wg, wu, X, act)
    bound = gated_bound(act, g, u, _sum_bound(wg, mg, X), _sum_bound(wu, mu, X))
    assert got.dtype == dtype and got.shape == (t, m)
    assert torch.all((got.double() - h).abs() <= bound * (1 + 2.0 ** -8) + half_step(dtype, h))


def test_products_shapes_strides_and_outputs():
    w = _random_weights(70, 200, 64, True, seed=3)
    big = _vectors(12, 450, 1, BF16)
    ref = ext.int4_matvec(w, big[:, 8:208].contiguous())
    for view in (big[:, 8:208], big[::1, 8:208]):
        assert torch.equal(ext.int4_matvec(w, view), ref)
    odd = ext.int4_matvec(w, big[:, 7:207])                     # rows off every 16-byte boundary
    assert torch.equal(odd, ext.int4_matvec(w, big[:, 7:207].contiguous()))
    assert torch.equal(ext.int4_matvec(w, big[3, 8:208]), ref[3])
    out = torch.full((14, 90), 7.0, dtype=BF16, device="cuda")
    got = ext.int4_matvec(w, big[:, 8:208], out=out[1:13, 11:81])
    assert got.data_ptr() == out[1:13, 11:81].data_ptr() and torch.equal(got, ref)
    rest = out.clone()
    rest[1:13, 11:81] = 7.0
    assert torch.all(rest == 7.0)                               # nothing beside the result is written
    assert ext.int4_matvec(w, big[:0, 8:208]).shape == (0, 70)
    assert ext.int4_gated(w, w, big[:0, 8:208]).shape == (0, 70)


def test_products_take_any_leading_dimensions():
    """(batch, sequence, n) and more, as the dense block does; each row as in a call with two dimensions."""
    w = _random_weights(70, 200, 64, True, seed=4)
    X = _vectors(24, 200, 2, BF16)
    y, h = ext.int4_matvec(w, X), ext.int4_gated(w, w, X)
    for lead in ((4, 6), (2, 3, 4), (1, 24)):
        assert torch.equal(ext.int4_matvec(w, X.view(*lead, 200)), y.view(*lead, 70))
        assert torch.equal(ext.int4_gated(w, w, X.view(*lead, 200)), h.view(*lead, 70))
    out = torch.zeros(4, 6, 70, dtype=BF16, device="cuda")
    got = ext.int4_matvec(w, X.view(6, 4, 200).transpose(0, 1), out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, y.view(6, 4, 70).transpose(0, 1))
    one = torch.zeros(70, dtype=BF16, device="cuda")
    assert ext.int4_matvec(w, X[0], out=one).shape == (70,) and torch.equal(one, ext.int4_matvec(w, X[0]))
    assert ext.int4_matvec(w, X.view(4, 6, 200)[:0]).shape == (0, 6, 70)
    for bad, kw in ((X[:, :199], {}), (X[0, 0], {}), (X, dict(out=out)), (X.view(4, 6, 200), dict(out=out[:, :5])), (X[0], dict(out=[0])),
                    (X[0], dict(out=torch.zeros(140, dtype=BF16, device="cuda")[::2])), (X, dict(out=y.float()))):
        with pytest.raises(ValueError):
            ext.int4_matvec(w, bad, **kw)
    with pytest.raises(ValueError, match="last dimension must be 200"):
        ext.int4_matvec(w, X.view(4, 6, 200)[..., :100])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_rows_do_not_influence_one_another(dtype):
    w = _random_weights(40, 300, 64, True, seed=9)
    X = _vectors(20, 300, 9, dtype)
    ref = ext.int4_matvec(w, X)
    X[4] = float("nan")
    X[11, 7] = float("inf")
    got = ext.int4_matvec(w, X)
    keep = [i for i in range(20) if i not in (4, 11)]
    assert torch.equal(got[keep], ref[keep])
    assert torch.isnan(got[4]).all() and not torch.isfinite(got[11]).any()


def test_fp32_vectors_of_huge_and_tiny_range():
    w = _random_weights(40, 300, 64, True, seed=10)
    X = _vectors(4, 300, 10, F32)
    X[1] *= 2.0 ** 105
    X[2] *= 2.0 ** -90
    W, mag = _values64(w)
    y = X.double() @ W.t()
    got = ext.int4_matvec(w, X).double()
    assert torch.all((got - y).abs() <= _sum_bound(w, mag, X) * (1 + 2.0 ** -8) + half_step(F32, y))


@pytest.mark.parametrize("t", [4, 20])
def test_fp32_vectors_near_the_end_of_the_range(t):
    """The third of an entry's three terms ends at bf16's least subnormal, 2^-133: what lies below it is lost."""
    w = _random_weights(40, 300, 64, True, seed=10)
    w.scale.fill_(1.0)
    W, mag = _values64(w)
    for e in (100, 112, 120, 126, 132, 140):
        X = (_vectors(t, 300, 10, F32).double() * 2.0 ** -e).float()
        y = X.double() @ W.t()
        got = ext.int4_matvec(w, X).double()
        lost = 2.0 ** -133 * mag.sum(1)
        assert torch.all((got - y).abs() <= (_sum_bound(w, mag, X) + lost) * (1 + 2.0 ** -8) + half_step(F32, y))


def test_products_repeat_bit_for_bit_on_streams_and_in_graphs():
    w = _random_weights(500, 1300, 128, True, seed=12)
    X = _vectors(24, 1300, 12, F16)
    ref_y, ref_h = ext.int4_matvec(w, X), ext.int4_gated(w, w, X, "gelu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        y, h = ext.int4_matvec(w, X, stream=s), ext.int4_gated(w, w, X, "gelu", stream=s.cuda_stream)
        s.synchronize()
        assert torch.equal(y, ref_y) and torch.equal(h, ref_h)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    A = _matrix(50, 700, 2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, h = ext.int4_matvec(w, X), ext.int4_gated(w, w, X, "gelu")
        wq = ext.int4_quantize(A, 64, async_status=st)
        v = ext.int4_dequantize(wq)
    for _ in range(2):
        y.zero_(), h.zero_(), v.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref_y) and torch.equal(h, ref_h)
        assert torch.equal(v, ext.int4_dequantize(ext.int4_quantize(A, 64)))


@pytest.mark.parametrize("blocks", range(1, 12))
def test_every_share_of_the_columns(blocks):
    """More than 8 vectors split a tile's columns over 1 to 8 CTAs, whose sums meet in a fixed order."""
    n = 128 * blocks - 5
    w, X = _random_weights(150, n, 32, True, seed=blocks), _vectors(20, n, blocks, F16)
    W, mag = _values64(w)
    y = X.double() @ W.t()
    got = ext.int4_matvec(w, X)
    assert torch.all((got.double() - y).abs() <= _sum_bound(w, mag, X) * (1 + 2.0 ** -8) + half_step(F16, y))
    assert torch.equal(got, ext.int4_matvec(w, X))


@pytest.mark.parametrize("t,m,n", [(9, 100, 100), (20, 300, 2000), (64, 1000, 1500)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_waits_that_run_out_leave_nan(t, m, n, dtype):
    """The products of one CTA are withheld (a host-set flag): its waits give up and its tile is NaN, the others' tiles
    are right, and so is the next call."""
    w, X = _random_weights(m, n, 64, True, seed=t), _vectors(t, n, t, dtype)
    ref, href = ext.int4_matvec(w, X), ext.int4_gated(w, w, X)
    with ext.debug_wait_fault(1):
        y, h = ext.int4_matvec(w, X), ext.int4_gated(w, w, X)
    for got, want, rows in ((y, ref, 128), (h, href, 64)):
        assert torch.isnan(got[:, :rows]).all() and torch.equal(got[:, rows:], want[:, rows:])
    assert torch.equal(ext.int4_matvec(w, X), ref) and torch.equal(ext.int4_gated(w, w, X), href)


def test_calls_on_two_streams_at_once():
    w, big = _random_weights(700, 2000, 64, True, seed=1), _random_weights(3000, 1024, 128, False, seed=2)
    X, Z = _vectors(30, 2000, 1, BF16), _vectors(5, 1024, 2, F32)
    ref, ref2 = ext.int4_matvec(w, X), ext.int4_matvec(big, Z)
    torch.cuda.synchronize()
    s, r = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(20):
        outs.append((ext.int4_matvec(w, X, stream=s), ext.int4_matvec(big, Z, stream=r), ext.int4_gated(w, w, X, stream=r)))
    torch.cuda.synchronize()
    h = ext.int4_gated(w, w, X)
    assert all(torch.equal(a, ref) and torch.equal(b, ref2) and torch.equal(c, h) for a, b, c in outs)


def test_matrices_past_32_bit_offsets():
    """Codes of more than 4 GiB: the last rows are the last rows."""
    m, n, group = 70001, 131072, 128
    q = torch.randint(0, 256, (m, ext.int4_row_bytes(n)), dtype=torch.uint8, device="cuda")
    s = torch.rand(n // group, m, device="cuda").half() * 0.01
    w = ext.Int4Weights(q, s, None, m, n, group)
    tail = ext.Int4Weights(q[-40:].clone(), s[:, -40:].contiguous(), None, 40, n, group)
    # (a large matrix is split into other shares than a small one, so the rows are compared with 64 bits)
    W, mag = _values64(tail)
    for t in (1, 12):
        X = _vectors(t, n, t, F16)
        y = X.double() @ W.t()
        got = ext.int4_matvec(w, X)[:, -40:].double()
        assert torch.all((got - y).abs() <= _sum_bound(tail, mag, X) * (1 + 2.0 ** -8) + half_step(F16, y))
    del q, w
    A = torch.zeros(40001, 65536, dtype=F16, device="cuda")          # 2.6 G entries, 5 GB
    A[-3:] = _matrix(3, 65536, 1, F16)
    w = ext.int4_quantize(A, 128)
    ref = ext.int4_quantize(A[-3:].clone(), 128)
    assert torch.equal(w.q[-3:], ref.q) and torch.equal(w.scale[:, -3:], ref.scale) and torch.equal(w.offset[:, -3:], ref.offset)
    v = ext.int4_dequantize(w, F16)
    assert torch.equal(v[-3:], ext.int4_dequantize(ref, F16)) and not v[:-3].any()


def test_library_refuses_bad_arguments():
    L, einval = ext._lib.load(), ext.STATUS["EINVAL"]
    w = _random_weights(20, 100, 64, True, seed=1)
    X, Y = _vectors(12, 104, 1, BF16), torch.zeros(12, 20, dtype=BF16, device="cuda")
    work = torch.zeros(L.externd_aligned_bytes(2, 11, 100), dtype=torch.uint8, device="cuda")
    base = dict(work=None, wb=0, q=w.q.data_ptr(), s=w.scale.data_ptr(), b=w.offset.data_ptr(), m=20, n=100, group=64, x=X.data_ptr(), dt=2,
                ldx=104, batch=3, y=Y.data_ptr(), ldy=20)

    def call(**kw):
        a = dict(base, **kw)
        return L.externd_int4_matvec(a["q"], a["s"], a["b"], a["m"], a["n"], a["group"], a["x"], a["dt"], a["ldx"], a["batch"],
                                     a["y"], a["ldy"], a["work"], a["wb"], torch.cuda.current_stream().cuda_stream)

    assert call() == 0
    host = torch.zeros(4096, dtype=torch.uint8)
    for kw in (dict(q=None), dict(s=None), dict(x=None), dict(y=None), dict(m=0), dict(n=0), dict(group=16), dict(group=256),
               dict(dt=3), dict(dt=-1), dict(ldx=99), dict(ldy=19), dict(batch=-1), dict(q=w.q.data_ptr() + 8),
               dict(s=w.scale.data_ptr() + 1), dict(x=X.data_ptr() + 1), dict(x=host.data_ptr()), dict(q=host.data_ptr())):
        assert call(**kw) == einval, kw
    assert call(batch=0, x=None, y=None) == 0
    # more than 8 rows off the 16-byte boundaries take their place in work
    assert call(x=X.data_ptr() + 2) == 0
    off = dict(x=X.data_ptr() + 2, batch=11)
    assert call(**off) == einval and call(**off, work=work.data_ptr(), wb=work.numel() - 1) == einval
    assert call(**off, work=host.data_ptr(), wb=work.numel()) == einval and call(**off, work=work.data_ptr() + 16, wb=work.numel()) == einval
    assert call(**off, work=work.data_ptr(), wb=work.numel()) == 0
