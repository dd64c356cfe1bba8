"""The block norms' and 4-bit calls' refusals without a GPU: status codes of the C ABI
before any HIP call (pointers are fake addresses), workspace queries, and the binding's
checks of devices, types, shapes and strides."""
import ctypes

import pytest
import torch

from mixture_experts_layer_16_amd import binding as B

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = ctypes.c_void_p(0x10000)
Y = ctypes.c_void_p(1 << 21)
MIS = ctypes.c_void_p(0x10002)


def norm(**kw):
    a = dict(T=8, d=128, k=0, dtype=1, x=P, y=P, y_perm=None, n_rows=0, slot_row=None, topk_w=None, post_gain=P,
             gate=None, gate_rows=0, gate_act=0, rs=1.0, bs=1.0, eps=1e-6, next_gain=P, out=P, h=P, y_out=None,
             stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return B.lib().moe_block_norm(*a.values())


PERM = dict(y=None, y_perm=P, k=2, n_rows=16, slot_row=P, topk_w=P)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(T=0)), (INVALID, dict(T=-1)), (INVALID, dict(d=0)), (UNSUPPORTED, dict(d=100)),
    (UNSUPPORTED, dict(d=16448)), (UNSUPPORTED, dict(T=1 << 31)), (UNSUPPORTED, dict(dtype=2)),
    (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))), (INVALID, dict(gate_act=3)),
    (INVALID, dict(gate=P)), (INVALID, dict(gate=P, gate_rows=-1)), (INVALID, dict(gate_rows=4)),
    (INVALID, dict(x=None)), (INVALID, dict(x=MIS)), (INVALID, dict(y=MIS)), (INVALID, dict(post_gain=MIS)),
    (INVALID, dict(next_gain=MIS)), (INVALID, dict(out=None)), (INVALID, dict(h=None)), (INVALID, dict(next_gain=None)),
    (INVALID, dict(k=2)), (INVALID, dict(slot_row=P)), (INVALID, dict(topk_w=P)), (INVALID, dict(y_out=P)),
    (INVALID, dict(n_rows=4)), (INVALID, dict(PERM, y=P)), (INVALID, dict(PERM, k=0)), (INVALID, dict(PERM, n_rows=0)),
    (INVALID, dict(PERM, slot_row=None)), (INVALID, dict(PERM, topk_w=None)), (INVALID, dict(PERM, y_out=MIS)),
    (UNSUPPORTED, dict(PERM, T=1 << 30, k=2)), (UNSUPPORTED, dict(PERM, n_rows=1 << 31)),
    (UNSUPPORTED, dict(PERM, k=1 << 62)),
    (INVALID, dict(y=None)), (INVALID, dict(y=None, post_gain=None)), (INVALID, dict(y=None, out=None)),
    (INVALID, dict(y=None, post_gain=None, out=None, next_gain=None, h=None)),
    (INVALID, dict(y=None, post_gain=None, out=None, gate=P, gate_rows=1))])
def test_block_norm_refuses(want, kw):
    assert norm(**kw) == want


def back(query=False, **kw):
    n = ctypes.c_size_t(1 << 40)
    a = dict(T=8, d=128, dtype=1, y=P, post_gain=P, gate=None, gate_rows=0, gate_act=0, rs=1.0, bs=1.0, eps=1e-6,
             out=P, next_gain=P, d_out=P, dh=P, dx=P, dy=P, d_post_gain=P, dgate=None, d_next_gain=P, ws=P,
             n=ctypes.byref(n), stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    if query:
        a["ws"] = None
    st = B.lib().moe_block_norm_backward(*a.values())
    return (st, n.value) if query else st


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(T=0)), (UNSUPPORTED, dict(d=96)), (UNSUPPORTED, dict(d=1 << 15)), (UNSUPPORTED, dict(dtype=7)),
    (INVALID, dict(eps=-1e-9)), (INVALID, dict(gate_act=-1)), (INVALID, dict(gate=P)), (INVALID, dict(gate_rows=1)),
    (INVALID, dict(gate=P, gate_rows=1)), (INVALID, dict(dgate=P)), (INVALID, dict(dx=None)), (INVALID, dict(dx=MIS)),
    (INVALID, dict(dy=None)), (INVALID, dict(y=None)), (INVALID, dict(y=None, dy=None)),
    (INVALID, dict(post_gain=None)), (INVALID, dict(d_post_gain=None)), (INVALID, dict(out=None)),
    (INVALID, dict(dh=None)), (INVALID, dict(d_next_gain=None)), (INVALID, dict(next_gain=None)),
    (INVALID, dict(out=None, dh=None, next_gain=None, d_next_gain=None, d_out=None)),
    (INVALID, dict(d_out=MIS)), (INVALID, dict(dh=MIS)), (INVALID, dict(ws=MIS)), (WORKSPACE, dict(ws=None, n=None)),
    (WORKSPACE, dict(n=ctypes.byref(ctypes.c_size_t(256))))])
def test_block_norm_backward_refuses(want, kw):
    assert back(**kw) == want


def test_block_norm_backward_workspace():
    # one part of d floats for a workgroup and sum; two rows a team at least (one, where 128 workgroups
    # then do), and 12 wavefronts' teams for 256 CUs at most: 24,576 (d <= 64, 32 a workgroup), 12,288
    # (<= 128, 16), 6,144 (<= 256, 8), half of it (<= 512, 4), 1,536 (<= 1,024, 1 as from here on),
    # 1,024 (<= 1,536), 768 (<= 2,048)
    assert back(query=True) == (OK, 2 * 1 * 128 * 4)
    assert back(query=True, next_gain=None) == (OK, 1 * 128 * 4)
    assert back(query=True, T=2, d=1024) == (OK, 2 * 1 * 1024 * 4)
    assert back(query=True, T=3, d=1024) == (OK, 2 * 3 * 1024 * 4)
    assert back(query=True, T=128, d=1024) == (OK, 2 * 128 * 1024 * 4)
    assert back(query=True, T=129, d=1024) == (OK, 2 * 65 * 1024 * 4)
    assert back(query=True, post_gain=None, next_gain=None) == (OK, 0)
    assert back(query=True, T=4096, d=1024) == (OK, 2 * 1366 * 1024 * 4)
    assert back(query=True, T=4096, d=2048) == (OK, 2 * 683 * 2048 * 4)
    # 2,048 rows a gate group, 6 rows a team: 342 teams a group and their own parts
    assert back(query=True, T=4096, d=2048, gate=P, gate_rows=2048) == (OK, 3 * 684 * 2048 * 4)
    assert back(query=True, T=4096, d=1088) == (OK, 2 * 1024 * 1088 * 4)
    # one group, of T rows or any number above
    for rows in (4096, 4097, 2 ** 63 - 1):
        assert back(query=True, T=4096, d=2048, gate=P, gate_rows=rows) == (OK, 3 * 683 * 2048 * 4)
    assert back(query=True, T=1, gate=P, gate_rows=2 ** 63 - 1) == back(query=True, T=1, gate=P, gate_rows=2)
    # groups of 4 rows: 8 rows a team, no parts of the gate
    assert back(query=True, T=4096, d=2048, gate=P, gate_rows=4) == (OK, 2 * 512 * 2048 * 4)
    # narrow rows, 9 a team: 22,223 teams; groups of 36 are still a team's; groups of 100 have 12
    # teams with parts of their own, groups of 5,963 have 663, made 21 workgroups, with one each
    assert back(query=True, T=200000, d=64) == (OK, 2 * 695 * 64 * 4)
    assert back(query=True, T=200000, d=64, gate=P, gate_rows=36) == (OK, 2 * 174 * 64 * 4)
    assert back(query=True, T=200000, d=64, gate=P, gate_rows=100) == (OK, (2 * 750 + 24000) * 64 * 4)
    assert back(query=True, T=200000, d=64, gate=P, gate_rows=5963) == (OK, (2 * 714 + 714) * 64 * 4)


def w4(fn, **kw):
    a = {"moe_w4_quantize": dict(n=2, R=64, C=128, dtype=1, group=64, w=P, codes=P, scales=P, stream=None),
         "moe_w4_pack": dict(n=2, R=64, C=128, group=64, q=P, s=P, codes=P, scales=P, stream=None),
         "moe_w4_dequantize": dict(n=2, R=64, C=128, dtype=1, group=64, codes=P, scales=P, w=P, stream=None)}[fn]
    a.update(kw)
    return getattr(B.lib(), fn)(*a.values())


@pytest.mark.parametrize("fn", ["moe_w4_quantize", "moe_w4_pack", "moe_w4_dequantize"])
@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(n=0)), (INVALID, dict(R=0)), (INVALID, dict(C=-32)), (UNSUPPORTED, dict(group=16)),
    (UNSUPPORTED, dict(group=0)), (UNSUPPORTED, dict(C=100)), (UNSUPPORTED, dict(C=1 << 21)),
    (UNSUPPORTED, dict(R=(1 << 20) + 1)), (UNSUPPORTED, dict(n=1 << 60)), (UNSUPPORTED, dict(n=1 << 25, C=256)),
    (INVALID, dict(codes=None)), (INVALID, dict(codes=MIS)), (INVALID, dict(scales=None)), (INVALID, dict(scales=MIS))])
def test_w4_layout_calls_refuse(fn, want, kw):
    assert w4(fn, **kw) == want


def test_w4_layout_calls_refuse_their_own():
    assert w4("moe_w4_quantize", w=None) == INVALID and w4("moe_w4_dequantize", w=MIS) == INVALID
    assert w4("moe_w4_pack", q=None) == INVALID and w4("moe_w4_pack", s=MIS) == INVALID
    assert w4("moe_w4_quantize", dtype=2) == UNSUPPORTED and w4("moe_w4_dequantize", dtype=-1) == UNSUPPORTED


def matvec(**kw):
    n = ctypes.c_size_t(1 << 40)
    a = dict(T=3, C=128, R=64, dtype=0, group=128, x=P, codes=P, scales=P, y=Y, ws=P, n=ctypes.byref(n), stream=None)
    a.update(kw)
    return B.lib().moe_w4_matvec(*a.values()), n.value


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(T=0)), (INVALID, dict(R=0)), (UNSUPPORTED, dict(C=48)), (UNSUPPORTED, dict(group=256)),
    (UNSUPPORTED, dict(dtype=3)), (UNSUPPORTED, dict(T=(1 << 19) + 1)), (UNSUPPORTED, dict(T=1 << 19, R=8192)),
    (UNSUPPORTED, dict(T=1 << 15, C=1 << 20)), (UNSUPPORTED, dict(T=1 << 11, C=1 << 20, dtype=1)), (INVALID, dict(x=None)), (INVALID, dict(x=MIS)),
    (INVALID, dict(codes=MIS)), (INVALID, dict(scales=None)), (INVALID, dict(y=None)), (INVALID, dict(y=P)), (INVALID, dict(ws=MIS)),
    (WORKSPACE, dict(ws=None, n=None)), (WORKSPACE, dict(n=ctypes.byref(ctypes.c_size_t(64))))])
def test_matvec_refuses(want, kw):
    assert matvec(**kw)[0] == want


def test_matvec_workspace():
    assert matvec(ws=None) == (OK, 3 * 128 * 6)
    assert matvec(ws=None, dtype=1) == (OK, 0)


def ffn(**kw):
    n = ctypes.c_size_t(1 << 40)
    a = dict(n_max=8, d=128, E=4, F=64, dtype=1, group=32, x=P, n_in=5, a_rows=P, offsets=P, gc=P, gs=P, uc=P, us=P,
             dc=P, ds=P, y=P, ws=P, n=ctypes.byref(n), stream=None)
    a.update(kw)
    return B.lib().moe_w4_grouped_ffn(*a.values()), n.value


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(n_max=0)), (INVALID, dict(E=0)), (UNSUPPORTED, dict(E=1025)), (UNSUPPORTED, dict(d=96)),
    (UNSUPPORTED, dict(F=32)), (UNSUPPORTED, dict(group=48)), (UNSUPPORTED, dict(dtype=2)), (INVALID, dict(n_in=0)),
    (UNSUPPORTED, dict(n_in=1 << 31)), (UNSUPPORTED, dict(n_in=1 << 24)), (UNSUPPORTED, dict(n_max=(1 << 19) + 1)),
    (UNSUPPORTED, dict(n_max=1 << 19, d=1 << 14)), (UNSUPPORTED, dict(n_max=1 << 15, F=1 << 16)), (UNSUPPORTED, dict(E=1024, d=1 << 13, F=1 << 14)),
    (INVALID, dict(offsets=None)), (INVALID, dict(x=None)), (INVALID, dict(gc=MIS)), (INVALID, dict(gs=None)),
    (INVALID, dict(uc=None)), (INVALID, dict(us=MIS)), (INVALID, dict(dc=None)), (INVALID, dict(ds=None)),
    (INVALID, dict(y=MIS)), (INVALID, dict(ws=MIS)), (WORKSPACE, dict(ws=None, n=None)),
    (WORKSPACE, dict(n=ctypes.byref(ctypes.c_size_t(256))))])
def test_grouped_ffn_refuses(want, kw):
    assert ffn(**kw)[0] == want


def test_grouped_ffn_workspace():
    assert ffn(ws=None) == (OK, 8 * 64 * 4)
    assert ffn(ws=None, dtype=0) == (OK, 8 * 64 * 6 + 5 * 128 * 6)
    assert ffn(ws=None, dtype=0, a_rows=None, n_in=0) == (OK, 8 * 64 * 6 + 8 * 128 * 6)


# ---- the binding's own checks (CPU tensors: refused before the library is called) ----

def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("err,kw", [
    (ValueError, dict(y=t(4, 64))), (TypeError, dict(y=t(5, 64, dtype=torch.float32))),
    (ValueError, dict(y=t(5, 128)[:, ::2])), (TypeError, dict(next_gain=t(64))),
    (ValueError, dict(next_gain=t(63, dtype=torch.float32))),
    (ValueError, dict(y=t(5, 64), gate=t(2, 64), gate_rows=5)), (ValueError, dict(y=t(5, 64), gate=t(1, 64))),
    (ValueError, dict(y=t(5, 64), gate_act="relu")), (ValueError, dict(y_perm=t(10, 64))),
    (TypeError, dict(y_perm=t(10, 64), slot_row=t(5, 2), topk_w=t(5, 2))),
    (ValueError, dict(y=torch.zeros(5, 64, dtype=torch.bfloat16, device="meta")))])
def test_binding_refuses_norm_operands(err, kw):
    with pytest.raises(err):
        B.BlockNorm(t(5, 64), **kw)


@pytest.mark.parametrize("err,kw", [
    (ValueError, dict()), (ValueError, dict(d_out=t(5, 64), y=t(6, 64))),
    (TypeError, dict(d_out=t(5, 64), dh=t(5, 64, dtype=torch.float32))),
    (ValueError, dict(d_out=t(5, 64), y=t(5, 64), gate=t(3, 64), gate_rows=5)),
    (B.MoEError, dict(dh=t(5, 64)[:, :63].contiguous()))])
def test_binding_refuses_gradients(err, kw):
    with pytest.raises(err):
        B.BlockNormBackward(**kw)


def test_binding_refuses_weights():
    with pytest.raises(B.MoEError):
        B.W4Weights(1, 16, 128, 48, "cpu")
    w = B.W4Weights(2, 64, 128, 64, "cpu")
    one = B.W4Weights(1, 64, 128, 64, "cpu")
    with pytest.raises(ValueError):
        B.W4Matvec(t(3, 128), w)                            # two matrices
    with pytest.raises(ValueError):
        B.W4Matvec(t(3, 64), one)                           # other columns
    with pytest.raises(ValueError):
        B.moe_w4_pack(t(1, 4, 64, dtype=torch.uint8), t(1, 4, 1), 64)
    with pytest.raises(TypeError):
        B.moe_w4_pack(t(1, 4, 64, dtype=torch.uint8), t(1, 4, 2, dtype=torch.float32), 64)
    with pytest.raises(ValueError):
        w.dequantize(out=t(2, 64, 64))
    down = B.W4Weights(2, 128, 64, 64, "cpu")
    off = t(3, dtype=torch.int32)
    for kw in (dict(up=one), dict(down=w), dict(offsets=t(2, dtype=torch.int32)), dict(x_in=t(3, 64)), dict(n_max=9),
               dict(a_rows=t(4, dtype=torch.int32), n_max=5), dict(y_perm=t(4, 128))):
        with pytest.raises(ValueError):
            B.W4GroupedFfn(**dict(dict(x_in=t(3, 128), offsets=off, gate=w, up=w, down=down), **kw))
