"""Host-side checks of the 4-bit and gated feed-forward entry points: layouts, and refusals before any device
work."""
import ctypes

import numpy as np
import pytest
import torch

import ternary_rank_weight_b200 as ext
from ternary_rank_weight_b200 import _lib

EINVAL = ext.STATUS["EINVAL"]


def test_int4_layout_follows_its_rule():
    assert [ext.int4_row_bytes(n) for n in (0, 1, 128, 129, 6912)] == [0, 64, 64, 128, 3456]
    n = 300
    codes = np.random.default_rng(1).integers(0, 16, size=(5, n)).astype(np.uint8)
    packed = ext.pack_int4(codes)
    assert packed.shape == (5, ext.int4_row_bytes(n))
    assert np.array_equal(ext.unpack_int4(packed, n), codes)
    words = packed.view("<u4")
    for j in range(384):                                   # column 128 B + 32 i + 8 c + t, padding 8
        blk, i, c, t = j // 128, j // 32 % 4, j // 8 % 4, j % 8
        got = (words[:, 16 * blk + 4 * c + i] >> (4 * (4 * (t % 2) + t // 2))) & 15
        assert np.array_equal(got, codes[:, j] if j < n else np.full(5, 8)), j


def test_int4_entry_points_reject_bad_arguments_before_device_work():
    L = _lib.load()
    host = (ctypes.c_uint8 * 256)()
    p = (ctypes.addressof(host) + 15) // 16 * 16
    assert L.externd_int4_quantize(None, 0, 1, 1, 1, 32, p, p, None, None, None) == EINVAL
    assert L.externd_int4_quantize(p, 0, 1, 1, 1, 32, p, p, None, None, None) == EINVAL        # host memory
    assert L.externd_int4_quantize(p, 0, 0, 1, 1, 32, p, p, None, None, None) == EINVAL
    assert L.externd_int4_quantize(p, 0, 1, 4, 3, 32, p, p, None, None, None) == EINVAL        # lda < n
    assert L.externd_int4_quantize(p, 3, 1, 1, 1, 32, p, p, None, None, None) == EINVAL
    assert L.externd_int4_quantize(p, 0, 1, 1, 1, 48, p, p, None, None, None) == EINVAL
    assert L.externd_int4_dequantize(p, p, None, 1, 1, 32, p, 0, 1, None) == EINVAL            # host memory
    assert L.externd_int4_dequantize(p, p, None, 1, 1, 32, None, 0, 1, None) == EINVAL
    assert L.externd_int4_matvec(p, p, None, 1, 1, 32, p, 0, 1, 1, p, 1, None, 0, None) == EINVAL       # host memory
    assert L.externd_int4_matvec(p, p, None, 1, 1, 32, p, 0, 1, -1, p, 1, None, 0, None) == EINVAL
    assert L.externd_int4_gated(p, p, None, p, p, None, 1, 1, 32, 4, p, 0, 1, 1, p, 1, None, 0, None) == EINVAL   # activation


def test_int4_binding_rejects_bad_tensors():
    cpu = torch.zeros(4, 128)
    with pytest.raises(ValueError):
        ext.int4_quantize(cpu)                                       # not on the GPU
    with pytest.raises(ValueError):
        ext.int4_quantize(np.zeros((4, 128), dtype=np.float32))
    w = ext.Int4Weights(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.float16), None, 4, 128, 128)
    with pytest.raises(ValueError):
        ext.int4_dequantize(w)
    with pytest.raises(ValueError):
        ext.int4_matvec(w, cpu)
    with pytest.raises(ValueError):
        ext.int4_gated(w, w, cpu, "swish")
    with pytest.raises(ValueError):
        ext.int4_matvec(w, None)


def test_gated_entry_points_reject_bad_arguments_before_device_work():
    L = _lib.load()
    host = (ctypes.c_uint8 * 512)()
    p = (ctypes.addressof(host) + 255) // 256 * 256
    base = dict(x=p, w=p, dt=2, m=1, n=1, t=1, act=0, h=p, g=None, sd=0, wb=0, work=None)

    def fwd(**kw):
        a = dict(base, **kw)
        return L.externd_gated(a["x"], 8, p, 8, a["w"], 8, a["dt"], a["m"], a["n"], a["t"], a["act"], a["h"], 1, a["g"], a["g"],
                               a["sd"], 1, a["work"], a["wb"], None, None)

    for kw in ({}, dict(w=None), dict(dt=0), dict(act=9), dict(m=0), dict(n=0), dict(t=-1), dict(h=None), dict(wb=256)):
        assert fwd(**kw) == EINVAL, kw                                       # {}: host memory
    assert L.externd_gated_backward(p, 1, p, 8, p, 8, p, 8, p, p, 0, 1, 2, 1, 1, 1, 0, p, 1, p, p, 1, p, 512, None, None) == EINVAL
    assert L.externd_aligned_bytes(1, 0, 5) == 0 and L.externd_aligned_bytes(1, 5, 0) == 0 and L.externd_aligned_bytes(7, 5, 5) == 0
    assert L.externd_aligned_bytes(2, 3, 9) == 256 and L.externd_aligned_bytes(1, 100, 9) == 3328
    assert L.externd_aligned_bytes(0, 100, 9) == 4864                       # fp32: rows of 48 bytes
    assert L.externd_gated_backward_work(0, 5, 5) == 0 and L.externd_gated_backward_work(5, 5, 0) == 0
    # two planes of 8-element rows on 256 bytes; besides, with few tokens, shares of dX
    assert L.externd_gated_backward_work(3, 3, 1) == 512
    assert L.externd_gated_backward_work(1000, 2560, 4096) == 2 * 4096 * 1000 * 2
    assert L.externd_gated_backward_work(6912, 2560, 64) > 2 * 64 * 6912 * 2


def test_shared_memory_of_outputs_and_inputs_is_seen():
    from ternary_rank_weight_b200.api import _overlap
    buf = torch.zeros(20, 64, dtype=torch.bfloat16)
    for a, b, want in [(buf[:, :30], buf[:, 30:], False), (buf[:, 30:], buf[:, :30], False), (buf[:, :31], buf[:, 30:], True),
                       (buf[:, 30:], buf[:, :31], True), (buf, buf, True), (buf[:10], buf[10:], False), (buf[:11], buf[10:], True),
                       (buf[:10, 40:], buf[9:, :41], True), (buf[:10, 40:], buf[9:, :40], False), (buf[:9, 40:], buf[9:, :41], False),
                       (buf[3:4], buf[3:4, :5], True), (buf[3:4, :5], buf[3:4, 5:], False), (buf[::2], buf[1::2], False),   # rows in turn
                       (buf[:0], buf, False), (buf, torch.zeros_like(buf), False), (buf[2:3, :8], buf[:, 8:], True)]:
        assert _overlap(a, b) == want and _overlap(b, a) == want, (a.shape, b.shape)


def test_wait_fault_hook_checks_its_arguments():
    L = _lib.load()
    for limit, worker in ((-1.0, 0), (float("nan"), 0), (1e-6, 0), (2.5, 0), (float("inf"), 0), (0.1, -1)):
        assert L.externd_debug_wait_fault(limit, worker) == EINVAL
    with ext.debug_wait_fault(3):
        pass
    assert L.externd_debug_wait_fault(0.0, 0) == 0


def test_gated_binding_rejects_bad_tensors():
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(8, 16, dtype=torch.bfloat16)
    for args in ((x, w, w), (x[:, :8], w, w), (x, w, w[:4]), (None, w, w), (x, None, w), (x.float(), w.float(), w.float())):
        with pytest.raises(ValueError):
            ext.gated(*args)
    with pytest.raises(ValueError):
        ext.gated(x, w, w, "tanh")
    with pytest.raises(ValueError):
        ext.gated_backward(x, x, w, w, x, x)
