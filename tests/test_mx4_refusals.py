"""What the MXFP4 x MXFP4 expert calls refuse, on the host and before any
launch (addresses here are never dereferenced)."""
import ctypes

import pytest

from mixture_experts_routed_moe_amd import _lib

A = 1 << 20
NULL, SHAPE, DTYPE, WORKSPACE = 1, 2, 3, 5


def _tables(T=8, K=2, E=4):
    s = _lib.MoeTablesStruct()
    L = _lib.lib()
    assert L.moe_tables_bind(ctypes.byref(s), A, L.moe_tables_bytes(T, K, E, 32), T, K, E, 32) == 0
    return s


def _call(name, bound=True, T=8, **bad):
    L = _lib.lib()
    t = _tables(T) if bound else _lib.MoeTablesStruct()
    d = dict(a=A, sa=A, w=A, sw=A, H=256, D=256, dtype=1, out=A, out2=A, ws=A, n=1 << 40)
    d.update(bad)
    if name == "gate_up":
        return L.moe_expert_gate_up_mx4(d["a"], d["sa"], d["w"], d["w"], d["sw"], d["sw"], ctypes.byref(t), d["H"],
                                        d["D"], d["out"], d["out2"], None)
    if name == "down":
        return L.moe_expert_down_mx4(d["a"], d["sa"], d["w"], d["sw"], ctypes.byref(t), d["H"], d["D"], d["dtype"],
                                     d["out"], None)
    return L.moe_routed_forward_mx4(d["a"], d["w"], d["w"], d["w"], d["sw"], d["sw"], d["sw"], ctypes.byref(t),
                                    d["H"], d["D"], d["dtype"], d["ws"], d["n"], d["out"], None)


@pytest.mark.parametrize("name", ["gate_up", "down", "forward"])
@pytest.mark.parametrize("bad, status", [
    (dict(a=None), NULL), (dict(w=None), NULL), (dict(sw=None), NULL), (dict(out=None), NULL), (dict(bound=False), NULL),
    (dict(H=300), SHAPE), (dict(D=128), SHAPE), (dict(D=0), SHAPE), (dict(H=1 << 25), SHAPE),
    (dict(T=1 << 20, H=1 << 13), SHAPE), (dict(a=A + 8), SHAPE), (dict(w=A + 4), SHAPE), (dict(sw=A + 4), SHAPE),
    (dict(out=A + 2), SHAPE),
])
def test_refusals(name, bad, status):
    assert _call(name, **bad) == status
    assert _lib.lib().moe_last_error()


def test_more_refusals():
    assert _call("gate_up", sa=None) == NULL and _call("gate_up", out2=None) == NULL
    assert _call("down", sa=None) == NULL and _call("forward", ws=None) == NULL
    for dt in (2, 3, 7):
        assert _call("down", dtype=dt) == DTYPE and _call("forward", dtype=dt) == DTYPE
    f = _lib.lib().moe_forward_mx4_workspace_bytes
    need = f(8, 2, 256, 256, 1)
    assert need == 16 * 512 + 1024 + 256 + 2048 + 256      # expert_out, xq, xs, hq, hs
    assert _call("forward", n=need - 1) == WORKSPACE and _call("forward", ws=A + 16) == WORKSPACE
    assert f(0, 2, 256, 256, 1) == 0 and f(8, 2, 256, 256, 2) == 0
