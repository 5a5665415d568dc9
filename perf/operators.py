"""What is timed of the 4-bit weight and gated feed-forward operators.

Five kinds of pass, each as a user's program makes it:

* ``quantize``   a weight matrix (m x n) to 4 bits with one scale (and, affine, one offset) per row and
                 group of columns, and back to the values the 4 bits stand for;
* ``matvec``     Y = X W^T for ``tokens`` input vectors and 4-bit W;
* ``int4_gated`` H = act(X Wg^T) * (X Wu^T) with 4-bit Wg, Wu: the gated block while tokens are generated;
* ``gated``      the same with dense 16-bit weights: a single token, or a prompt;
* ``step``       the dense gated block in training: H, and from its gradient dH those of X, Wg and Wu.

A 4-bit weight is w = s (q - 8) + b with q in 0..15, s (and b) fp16 per row and group of columns.  With
``mn`` / ``mx`` the group's least and greatest entry and ``am`` its greatest magnitude,
    symmetric   s = am / 7,            b absent (0),
    affine      s = (mx - mn) / 15,    b = mn + 8 s   (s as stored),
s and b computed in 64 bits and rounded to 32, then 16 bits; q = clamp(rint((w - b) / s) + 8, 0, 15) with
the quotient in 64 bits and ties to even, and q = 8 where s = 0.

Storage: row r of q is ceil(n / 128) blocks of 64 bytes.  Column j = 128 B + 32 i + 8 c + t (i, c in 0..3,
t in 0..7) sits in block B, 32-bit word 4 c + i, nibble 4 (t % 2) + t // 2.  Padding columns hold 8.  Scales
and offsets are stored group by group: [ceil(n / group), m].
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # a small layer of a toy model, converted with the finest groups: launches count
        dict(name="quantize_256x256_g32_f32", kind="quantize", m=256, n=256, group=32, affine=False, dtype="f32"),
        # the MLP-shaped matrix of the factorization benchmark as a checkpoint holds it
        dict(name="quantize_2560x6912_g128_bf16", kind="quantize", m=2560, n=6912, group=128, affine=True,
             dtype="bf16"),
        # one generated token through the down projection of that MLP
        dict(name="matvec_1x2560x6912_g128_bf16", kind="matvec", tokens=1, m=2560, n=6912, group=128, affine=True,
             dtype="bf16"),
        # a few vectors in fp32 through an odd-sized layer with the finest groups
        dict(name="matvec_3x1000x777_g32_f32", kind="matvec", tokens=3, m=1000, n=777, group=32, affine=True,
             dtype="f32"),
        # one token through the widest projection of a large model: the weights alone fill the time
        dict(name="matvec_1x8192x28672_g128_f16", kind="matvec", tokens=1, m=8192, n=28672, group=128, affine=False,
             dtype="f16"),
        # a full decoding batch through a square attention projection
        dict(name="matvec_64x4096x4096_g64_bf16", kind="matvec", tokens=64, m=4096, n=4096, group=64, affine=True,
             dtype="bf16"),
        # one generated token through the gate and up projections
        dict(name="int4_gated_1x6912x2560_g128_bf16", kind="int4_gated", tokens=1, m=6912, n=2560, group=128,
             affine=False, act="silu", dtype="bf16"),
        # a batch of sequences through a ragged block
        dict(name="int4_gated_45x5461x2049_g64_f16", kind="int4_gated", tokens=45, m=5461, n=2049, group=64,
             affine=True, act="gelu", dtype="f16"),
        # one token through the unquantised block
        dict(name="gated_1x6912x2560_bf16", kind="gated", tokens=1, m=6912, n=2560, act="silu", dtype="bf16"),
        # a prompt of odd length
        dict(name="gated_1537x6912x2560_f16", kind="gated", tokens=1537, m=6912, n=2560, act="gelu_tanh",
             dtype="f16"),
        # a short, ragged training step
        dict(name="step_300x1111x777_f16", kind="step", tokens=300, m=1111, n=777, act="relu2", dtype="f16"),
        # a training step of ordinary length
        dict(name="step_4096x6912x2560_bf16", kind="step", tokens=4096, m=6912, n=2560, act="silu", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size, log-uniform; half of them rounded to a multiple of 64, the others as they fall."""
    v = _log(rng, lo, hi)
    return max(64, v // 64 * 64) if rng.random() < 0.5 else v


def draw(rng):
    kind = rng.choice(["quantize", "matvec", "int4_gated", "gated", "step"])
    c = dict(kind=kind)
    if kind == "quantize":
        c["m"], c["n"] = _size(rng, 64, 6912), _size(rng, 64, 6912)
        limit, per = 2560 * 6912, c["m"]
        c["n"] = max(1, min(c["n"], limit // per))
        c["dtype"] = rng.choice(["f32", "bf16", "f16"])
        if c["dtype"] == "f32":
            c["n"] = max(1, min(c["n"], limit // 2 // per))
    elif kind in ("matvec", "int4_gated"):
        c["tokens"] = _log(rng, 1, 64)
        c["m"], c["n"] = _size(rng, 128, 8192), _size(rng, 128, 28672 if kind == "matvec" else 8192)
        # neither more weights nor more arithmetic than the largest listed case of the kind
        if kind == "matvec":
            c["n"] = max(64, min(c["n"], 64 * 4096 * 4096 // (c["tokens"] * c["m"])))
        else:
            c["n"] = max(64, min(c["n"], 45 * 5461 * 2049 // (c["tokens"] * c["m"])))
        c["dtype"] = rng.choice(["f32", "bf16", "f16"])
    else:
        c["tokens"] = _log(rng, 1, 4096) if kind == "gated" else _log(rng, 64, 4096)
        c["m"], c["n"] = _size(rng, 256, 8192), _size(rng, 256, 4096)
        limit = 1537 * 6912 * 2560 if kind == "gated" else 4096 * 6912 * 2560
        c["n"] = max(64, min(c["n"], limit // (c["tokens"] * c["m"])))
        c["dtype"] = rng.choice(["bf16", "f16"])
    if kind in ("quantize", "matvec", "int4_gated"):
        c["group"], c["affine"] = rng.choice([32, 64, 128]), rng.random() < 0.5
    if kind in ("int4_gated", "gated", "step"):
        c["act"] = rng.choice(["silu", "gelu", "gelu_tanh", "relu2"])
    return c


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------

def _weight(gen, m, n):
    """Rows of log-normal scale and a few outlier columns, like trained projections."""
    w = torch.randn(m, n, generator=gen, device="cuda")
    w *= 0.02 * torch.exp(0.5 * torch.randn(m, 1, generator=gen, device="cuda"))
    cols = torch.randint(0, n, (min(8, n),), generator=gen, device="cuda")
    w[:, cols] *= 5.0
    return w


def _codes(gen, m, n, case):
    """A 4-bit matrix as a quantiser leaves it: packed codes, scales and offsets."""
    group = case["group"]
    blocks, groups = (n + 127) // 128, (n + group - 1) // group
    # codes of a normal group: bell-shaped around 8
    q = (torch.randn(m, blocks * 128, generator=gen, device="cuda") * 2.7 + 8).round().clamp(0, 15).to(torch.int32)
    q[:, n:] = 8
    s = (0.007 * torch.exp(0.5 * torch.randn(groups, m, generator=gen, device="cuda"))).to(torch.float16)
    b = None
    if case["affine"]:
        b = (0.004 * torch.randn(groups, m, generator=gen, device="cuda")).to(torch.float16)
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device="cuda", dtype=torch.int64)
    words = (q.view(m, blocks, 4, 4, 8).to(torch.int64) << shift).sum(-1)     # [m, B, i, c]
    words = words.transpose(2, 3).reshape(m, blocks * 16)                     # word 4 c + i
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    return words.view(torch.uint8).reshape(m, blocks * 64).contiguous(), s, b


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind, dt = case["kind"], _DT[case["dtype"]]
    m, n = case["m"], case["n"]
    if kind == "quantize":
        return {"A": _weight(gen, m, n).to(dt)}
    x = torch.randn(case["tokens"], n, generator=gen, device="cuda")
    x[:, torch.randint(0, n, (min(4, n),), generator=gen, device="cuda")] *= 4.0    # a few hot channels
    d = {"X": x.to(dt)}
    if kind == "matvec":
        d["q"], d["s"], d["b"] = _codes(gen, m, n, case)
    elif kind == "int4_gated":
        d["qg"], d["sg"], d["bg"] = _codes(gen, m, n, case)
        d["qu"], d["su"], d["bu"] = _codes(gen, m, n, case)
    else:
        d["Wg"], d["Wu"] = _weight(gen, m, n).to(dt), _weight(gen, m, n).to(dt)
        if kind == "step":
            d["dH"] = (0.01 * torch.randn(case["tokens"], m, generator=gen, device="cuda")).to(dt)
    return d


def prepare(case, seed):
    st = dict(case=case, **_inputs(case, seed))
    if own:
        import ternary_rank_weight_b200 as ext
        st["ext"] = ext
        m, n, g = case["m"], case["n"], case.get("group")
        if case["kind"] == "quantize":
            st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        elif case["kind"] == "matvec":
            st["w"] = ext.Int4Weights(st["q"], st["s"], st["b"], m, n, g)
        elif case["kind"] == "int4_gated":
            st["wg"] = ext.Int4Weights(st["qg"], st["sg"], st["bg"], m, n, g)
            st["wu"] = ext.Int4Weights(st["qu"], st["su"], st["bu"], m, n, g)
    return st


# ---------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------

def _act(name, g):
    """The activation and its derivative."""
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    if name == "gelu":
        c = 0.5 * (1.0 + torch.erf(g * 0.5 ** 0.5))
        return g * c, c + g * torch.exp(-0.5 * g * g) * (2.0 * math.pi) ** -0.5
    if name == "gelu_tanh":
        k = (2.0 / math.pi) ** 0.5
        t = torch.tanh(k * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3.0 * 0.044715 * g * g)
    r = torch.clamp(g, min=0.0)
    return r * r, 2.0 * r


def _values(q, s, b, n, group):
    """The weights that codes, scales and offsets stand for, in fp32."""
    m = q.shape[0]
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=q.device, dtype=torch.int32)
    w = q.view(torch.int32).view(m, -1, 4, 4).transpose(2, 3).reshape(m, -1, 1)
    w = ((w >> shift) & 15).reshape(m, -1)[:, :n].float() - 8.0
    w *= s.float().t().repeat_interleave(group, 1)[:, :n]
    if b is not None:
        w += b.float().t().repeat_interleave(group, 1)[:, :n]
    return w


def _quantize(a, group, affine):
    m, n = a.shape
    groups = (n + group - 1) // group
    x = torch.zeros(m, groups * group, dtype=torch.float64, device=a.device)
    x[:, :n] = a.double()
    if groups * group > n:                       # the last group's missing columns repeat its first
        x[:, n:] = x[:, (groups - 1) * group:(groups - 1) * group + 1]
    x = x.view(m, groups, group)
    b = None
    if affine:
        mn, mx = x.amin(-1), x.amax(-1)
        s = ((mx - mn) / 15.0).float().half()
        b = (mn + 8.0 * s.double()).float().half()
    else:
        s = (x.abs().amax(-1) / 7.0).float().half()
    sd = s.double().unsqueeze(-1)
    c = x if b is None else x - b.double().unsqueeze(-1)
    q = torch.where(sd == 0, torch.zeros_like(c), torch.round(c / sd)).clamp(-8.0, 7.0)
    w = q.float() * s.float().unsqueeze(-1)
    if b is not None:
        w += b.float().unsqueeze(-1)
    w = w.view(m, -1)[:, :n].to(a.dtype)
    return w, s.t().contiguous(), None if b is None else b.t().contiguous()


def run(st):
    case = st["case"]
    kind = case["kind"]
    if own:
        ext = st["ext"]
        if kind == "quantize":
            w = ext.int4_quantize(st["A"], case["group"], affine=case["affine"], async_status=st["status"])
            return [ext.int4_dequantize(w, st["A"].dtype), w.scale] + ([w.offset] if case["affine"] else [])
        if kind == "matvec":
            return ext.int4_matvec(st["w"], st["X"])
        if kind == "int4_gated":
            return ext.int4_gated(st["wg"], st["wu"], st["X"], case["act"])
        if kind == "gated":
            return ext.gated(st["X"], st["Wg"], st["Wu"], case["act"])
        h, g, u = ext.gated_forward(st["X"], st["Wg"], st["Wu"], case["act"])
        return [h, *ext.gated_backward(st["dH"], st["X"], st["Wg"], st["Wu"], g, u, case["act"])]
    if kind == "quantize":
        w, s, b = _quantize(st["A"], case["group"], case["affine"])
        return [w, s] + ([b] if case["affine"] else [])
    x = st["X"].float()
    dt = st["X"].dtype
    if kind == "matvec":
        return (x @ _values(st["q"], st["s"], st["b"], case["n"], case["group"]).t()).to(dt)
    if kind == "int4_gated":
        wg = _values(st["qg"], st["sg"], st["bg"], case["n"], case["group"])
        wu = _values(st["qu"], st["su"], st["bu"], case["n"], case["group"])
    else:
        wg, wu = st["Wg"].float(), st["Wu"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a, da = _act(case["act"], g)
    h = (a * u).to(dt)
    if kind != "step":
        return h
    dh = st["dH"].float()
    dg, du = dh * u * da, dh * a
    return [h, (dg @ wg + du @ wu).to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)]


def work(case):
    kind, m, n = case["kind"], case["m"], case["n"]
    e = _BYTES[case["dtype"]]
    if "group" in case:
        packed = m * n / 2 + m * ((n + case["group"] - 1) // case["group"]) * (4 if case["affine"] else 2)
    if kind == "quantize":
        # reads A, writes codes and scales, reads them back, writes the values
        return {"bytes": 2 * m * n * e + 2 * packed, "flops": 6 * m * n}
    t = case["tokens"]
    if kind == "matvec":
        return {"bytes": packed + t * (m + n) * e, "flops": 2 * t * m * n}
    if kind == "int4_gated":
        return {"bytes": 2 * packed + t * (m + n) * e, "flops": 4 * t * m * n}
    if kind == "gated":
        return {"bytes": (2 * m * n + t * (m + n)) * e, "flops": 4 * t * m * n}
    # X, Wg, Wu and dH read; H, dX, dWg, dWu written
    return {"bytes": (4 * m * n + 2 * t * (m + n)) * e, "flops": 12 * t * m * n}


# ---------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------

def _column_weights(q, s, b, n, group):
    """One column of the matrix after another, from the storage rule."""
    j = torch.arange(n, device=q.device)
    t, c, i, blk = j % 8, j // 8 % 4, j // 32 % 4, j // 128
    nib = 4 * (t % 2) + t // 2
    byte = 64 * blk + 4 * (4 * c + i) + nib // 2
    code = torch.bitwise_right_shift(q[:, byte].to(torch.int64), 4 * (nib % 2)) & 15
    k = j // group
    v = s.double()[k].t() * (code - 8)
    return v if b is None else v + b.double()[k].t()


def _gate64(name, z):
    if name == "silu":
        sg = torch.sigmoid(z)
        return z * sg, sg + z * sg * (1 - sg)
    if name == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        # (1 + tanh y) / 2 = sigmoid(2 y)
        sg = torch.sigmoid(2 * k * (z + 0.044715 * z ** 3))
        return z * sg, sg + 2 * k * z * sg * (1 - sg) * (1 + 0.134145 * z * z)
    pos = z > 0
    return torch.where(pos, z * z, 0.0), torch.where(pos, 2 * z, 0.0)


def exact(case, seed):
    d = _inputs(case, seed)
    kind, n, group = case["kind"], case["n"], case.get("group")
    if kind == "quantize":
        a = d["A"].double()
        val, scales, offs = [], [], []
        for k in range(0, n, group):
            col = a[:, k:k + group]
            if case["affine"]:
                lo, hi = col.min(1, keepdim=True)[0], col.max(1, keepdim=True)[0]
                s = ((hi - lo) / 15).to(torch.float32).to(torch.float16).double()
                b = (lo + 8 * s).to(torch.float32).to(torch.float16).double()
                offs.append(b[:, 0])
            else:
                s = (col.abs().max(1, keepdim=True)[0] / 7).to(torch.float32).to(torch.float16).double()
                b = torch.zeros_like(s)
            code = torch.where(s > 0, torch.round((col - b) / torch.where(s > 0, s, 1.0)), 0.0)
            val.append(b + s * torch.clamp(code, -8, 7))
            scales.append(s[:, 0])
        out = [torch.cat(val, 1), torch.stack(scales)]
        return out + [torch.stack(offs)] if case["affine"] else out
    x = d["X"].double()
    if kind == "matvec":
        return torch.einsum("tn,mn->tm", x, _column_weights(d["q"], d["s"], d["b"], n, group))
    if kind == "int4_gated":
        wg = _column_weights(d["qg"], d["sg"], d["bg"], n, group)
        wu = _column_weights(d["qu"], d["su"], d["bu"], n, group)
    else:
        wg, wu = d["Wg"].double(), d["Wu"].double()
    z, u = torch.einsum("tn,mn->tm", x, wg), torch.einsum("tn,mn->tm", x, wu)
    f, df = _gate64(case["act"], z)
    if kind != "step":
        return f * u
    r = d["dH"].double()
    gz, gu = r * df * u, r * f
    return [f * u, torch.einsum("tm,mn->tn", gz, wg) + torch.einsum("tm,mn->tn", gu, wu),
            torch.einsum("tm,tn->mn", gz, x), torch.einsum("tm,tn->mn", gu, x)]
