"""Refusals of the router's training operators and of the 4-bit integer
matrices, before any device work (CPU only)."""

import ctypes

import pytest
import torch

_lib_mod = pytest.importorskip("sparse_expert_execution_amd._lib")
from sparse_expert_execution_amd import ops  # noqa: E402

EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -4
FAKE = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def L():
    return _lib_mod.lib()


def _desc(**kw):
    base = dict(hidden=256, inter=128, n_experts=8, top_k=2)
    base.update(kw)
    return ctypes.byref(ops.make_desc(**base))


def _q4(rows=64, cols=256, group=128, zero=0):
    return ctypes.byref(_lib_mod.MoeQ4Desc(rows, cols, group, zero))


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), EINVAL), (dict(cols=0), EINVAL), (dict(rows=-5), EINVAL),
    (dict(rows=(1 << 24) + 1), EINVAL), (dict(cols=(1 << 20) + 1), EINVAL),
    (dict(rows=1 << 24, cols=1 << 20), EINVAL), (dict(group=16), EUNSUPPORTED),
    (dict(group=0), EUNSUPPORTED), (dict(zero=2), EINVAL)])
def test_q4_descriptors(L, kw, status):
    off, n = (ctypes.c_size_t * 3)(), ctypes.c_size_t()
    assert L.moe_q4_layout(_q4(**kw), off, ctypes.byref(n)) == status and L.moe_last_error()
    assert L.moe_q4_quantize(_q4(**kw), FAKE, 0, 1 << 21, FAKE, None) == status
    assert L.moe_q4_linear(_q4(**kw), FAKE, 1 << 21, 1, FAKE, FAKE, 0, 1 << 25, None) == status


def test_q4_layout_sizes(L):
    off, n = (ctypes.c_size_t * 3)(), ctypes.c_size_t()
    assert L.moe_q4_layout(_q4(17, 129, 32, 1), off, ctypes.byref(n)) == 0
    # 2 x 2 tiles, 8 groups of 32
    assert list(off) == [0, 4096, 4096 + 2 * 8 * 32] and n.value == 4096 + 2 * 8 * 48
    assert L.moe_q4_layout(_q4(17, 129, 32, 0), off, ctypes.byref(n)) == 0
    assert list(off) == [0, 4096, 0] and n.value == 4096 + 2 * 8 * 32
    assert L.moe_q4_layout(None, off, ctypes.byref(n)) == EINVAL
    assert L.moe_q4_layout(_q4(), None, ctypes.byref(n)) == EINVAL


def test_q4_calls(L):
    lin = L.moe_q4_linear
    assert lin(_q4(), None, 256, 1, FAKE, FAKE, 0, 64, None) == EINVAL
    assert lin(_q4(), FAKE, 256, 1, None, FAKE, 0, 64, None) == EINVAL
    assert lin(_q4(), FAKE, 256, 1, FAKE, None, 0, 64, None) == EINVAL
    assert lin(_q4(), FAKE, 255, 1, FAKE, FAKE, 0, 64, None) == EINVAL
    assert lin(_q4(), FAKE, 256, 1, FAKE, FAKE, 0, 63, None) == EINVAL
    assert lin(_q4(), FAKE, 256, -1, FAKE, FAKE, 0, 64, None) == EINVAL
    assert lin(_q4(), FAKE, 256, 65537, FAKE, FAKE, 0, 64, None) == EINVAL
    assert lin(_q4(), FAKE, 256, 1, FAKE, FAKE, 2, 64, None) == EUNSUPPORTED
    assert lin(_q4(), FAKE, 256, 1, ctypes.c_void_p(4104), FAKE, 0, 64, None) == EINVAL
    assert lin(_q4(), ODD, 256, 1, FAKE, FAKE, 0, 64, None) == EINVAL
    assert lin(_q4(), FAKE, 256, 1, FAKE, ctypes.c_void_p(4098), 0, 64, None) == EINVAL
    assert lin(_q4(), None, 0, 0, None, None, 0, 0, None) == 0            # T == 0
    assert L.moe_q4_quantize(_q4(), FAKE, 2, 256, FAKE, None) == EUNSUPPORTED
    assert L.moe_q4_quantize(_q4(), FAKE, 0, 255, FAKE, None) == EINVAL
    assert L.moe_q4_quantize(_q4(), None, 0, 256, FAKE, None) == EINVAL
    assert L.moe_q4_pack(_q4(), FAKE, FAKE, FAKE, FAKE, None) == EINVAL   # zeros without has_zero
    assert L.moe_q4_pack(_q4(zero=1), FAKE, FAKE, None, FAKE, None) == EINVAL
    assert L.moe_q4_pack(_q4(), FAKE, FAKE, None, ODD, None) == EINVAL


@pytest.mark.parametrize("wtype", ["int4_g32", "int4_g64", "int4_g128"])
def test_int4_experts(L, wtype):
    d = _desc(wtype=wtype)
    off, n = (ctypes.c_size_t * 6)(), ctypes.c_size_t()
    assert L.moe_expert_layout(d, off, ctypes.byref(n)) == 0
    g = int(wtype[6:])
    one = 256 * 128 // 2 + 256 * 128 // g * 2
    assert list(off) == [0, 16384, one, one + 16384, 2 * one, 2 * one + 16384]
    assert n.value == -(-3 * one // 256) * 256
    need = L.moe_workspace_bytes(d, 4, 1)
    assert need > 8192
    assert L.moe_decode_launch_tokens(d) == 64
    dec = lambda T, ws: L.moe_decode(d, FAKE, T, FAKE, FAKE, None, FAKE, None, FAKE, FAKE, ws, None)
    assert dec(4, need - 1) == EWORKSPACE
    assert dec(65, 1 << 40) == EINVAL
    assert dec(0, 0) == 0
    assert L.moe_prefill(d, FAKE, 4, FAKE, FAKE, None, FAKE, None, FAKE, FAKE, 1 << 40,
                         None) == EUNSUPPORTED
    assert L.moe_route_decode_noalloc(d, FAKE, FAKE, 1, FAKE, FAKE, None, FAKE, None, FAKE, None,
                                      None) == EUNSUPPORTED
    x = torch.zeros((1, 256), dtype=torch.bfloat16)
    ids, w = torch.zeros((1, 2), dtype=torch.int32), torch.zeros((1, 2))
    with pytest.raises(_lib_mod.MoeError) as e:
        ops.host_experts(ops.make_desc(256, 128, 8, 2, wtype=wtype), x, ids, w,
                         torch.zeros(8 * n.value, dtype=torch.uint8), torch.zeros((1, 256)))
    assert e.value.status == EUNSUPPORTED


def test_int4_decode_limits(L):
    d = _desc(n_experts=32, top_k=9, wtype="int4_g64")
    assert L.moe_decode(d, FAKE, 1, FAKE, FAKE, None, FAKE, None, FAKE, FAKE, 1 << 40,
                        None) == EUNSUPPORTED
    with pytest.raises(KeyError):
        ops.make_desc(256, 128, 8, 2, wtype="int4")


def test_gate_calls(L):
    need = L.moe_workspace_bytes(_desc(), 100, 3)
    assert need >= 100 // 16 * 8 * 8
    gate = L.moe_gate
    assert gate(_desc(), None, 4, None, FAKE, FAKE, None, None, None, 0, None) == EINVAL
    assert gate(_desc(), FAKE, 4, None, None, FAKE, None, None, None, 0, None) == EINVAL
    assert gate(_desc(), FAKE, 4, None, FAKE, None, None, None, None, 0, None) == EINVAL
    assert gate(_desc(), FAKE, -1, None, FAKE, FAKE, None, None, None, 0, None) == EINVAL
    assert gate(_desc(), FAKE, 100, None, FAKE, FAKE, FAKE, None, FAKE, need - 1,
                None) == EWORKSPACE
    assert gate(_desc(), FAKE, 100, None, FAKE, FAKE, None, FAKE, None, need, None) == EWORKSPACE
    assert gate(_desc(), FAKE, 100, None, FAKE, FAKE, None, FAKE, ODD, need, None) == EWORKSPACE
    assert gate(_desc(), None, 0, None, None, None, None, None, None, 0, None) == 0
    back = L.moe_gate_backward
    assert back(_desc(), FAKE, 4, FAKE, None, FAKE, None, None, FAKE, None) == EINVAL  # dw, no w
    assert back(_desc(), FAKE, 4, FAKE, FAKE, None, None, FAKE, FAKE, None) == EINVAL  # no counts
    assert back(_desc(), None, 4, FAKE, FAKE, None, None, None, FAKE, None) == EINVAL
    assert back(_desc(), FAKE, 4, FAKE, FAKE, None, None, None, None, None) == EINVAL
    assert back(_desc(), None, 0, None, None, None, None, None, None, None) == 0


def test_router_calls(L):
    assert L.moe_router_logits(_desc(), FAKE, FAKE, 4, None, None) == EINVAL
    assert L.moe_router_logits(_desc(), ODD, FAKE, 4, FAKE, None) == EINVAL
    assert L.moe_router_logits(_desc(), FAKE, FAKE, -4, FAKE, None) == EINVAL
    assert L.moe_router_logits(_desc(), None, None, 0, None, None) == 0
    need = L.moe_workspace_bytes(_desc(), 64, 4)
    back = L.moe_router_backward
    assert back(_desc(), FAKE, FAKE, 64, FAKE, FAKE, FAKE, FAKE, need - 1, None) == EWORKSPACE
    assert back(_desc(), FAKE, FAKE, 64, FAKE, FAKE, FAKE, None, need, None) == EWORKSPACE
    assert back(_desc(), FAKE, FAKE, 64, None, FAKE, FAKE, FAKE, need, None) == EINVAL
    assert back(_desc(), None, FAKE, 64, FAKE, FAKE, FAKE, FAKE, need, None) == EINVAL
    assert back(_desc(), FAKE, None, 64, FAKE, FAKE, FAKE, FAKE, need, None) == EINVAL
    assert back(_desc(), FAKE, FAKE, 64, FAKE, ODD, None, FAKE, need, None) == EINVAL
    assert back(_desc(), FAKE, FAKE, 64, FAKE, None, ODD, FAKE, need, None) == EINVAL
    assert back(_desc(), FAKE, FAKE, (1 << 20) + 1, FAKE, FAKE, None, FAKE, 1 << 50,
                None) == EUNSUPPORTED
    assert back(_desc(), None, None, 0, None, None, None, None, 0, None) == 0
    assert L.moe_workspace_bytes(_desc(), (1 << 20) + 1, 4) == 0
    assert L.moe_workspace_bytes(_desc(), 0, 4) > 0
    assert L.moe_workspace_bytes(_desc(), 0, 3) > 0


def test_router_gradients_that_overlap(L):
    """Each output against each of the others, by one byte at either end."""
    d = _desc()
    T, H, E = 64, d._obj.hidden, d._obj.n_experts
    size = dict(x=T * H * 2, w=E * H * 2, dz=T * E * 4, dx=T * H * 2, dw=E * H * 4)
    at = {n: (i + 1) << 32 for i, n in enumerate(size)}
    need = L.moe_workspace_bytes(d, T, 4)

    def call(p):
        return L.moe_router_backward(d, p["x"], p["w"], T, p["dz"], p["dx"], p["dw"], 1 << 40,
                                     need, None)
    for out in ("dx", "dw"):
        for other in size:
            if other != out:
                assert call({**at, out: at[other]}) == EINVAL
                assert call({**at, out: at[other] + size[other] - 16}) == EINVAL
                assert call({**at, out: at[other] - size[out] + 16}) == EINVAL


def test_python_checks_name_the_argument():
    d = ops.make_desc(256, 128, 8, 2)
    x = torch.zeros((3, 256), dtype=torch.bfloat16)
    wr = torch.zeros((8, 256), dtype=torch.bfloat16)
    z = torch.zeros((3, 8))
    with pytest.raises(ValueError, match="x is on cpu, not on the current device"):
        ops.router_logits(d, x, wr, z)
    with pytest.raises(TypeError, match="x must be"):
        ops.router_logits(d, x.float(), wr, z)
    with pytest.raises(ValueError, match="x must have shape"):
        ops.router_logits(d, x[:, :128], wr, z)
    with pytest.raises(ValueError, match="logits must be contiguous"):
        ops.gate(d, torch.zeros((8, 3)).t(), None, None)
    q = ops.make_q4(16, 32, group=32)
    with pytest.raises(ValueError, match="rows"):
        ops.q4_linear(q, torch.zeros((32, 4), dtype=torch.bfloat16).t(), None, None)
    with pytest.raises(TypeError, match="src"):
        ops.q4_quantize(q, torch.zeros((16, 32), dtype=torch.float16), None)
