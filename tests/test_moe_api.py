"""Host-side checks of the mixture-of-experts calls: workspaces, refusals, struct layouts.

Every call below fails a check that runs before the first CUDA call, or is an empty
problem, so no pointer here is ever dereferenced.
"""
import ctypes
import os
import subprocess

import moe_reference as ref
import numpy as np
import pytest

import gemm_decode_gb300 as q4
from gemm_decode_gb300 import build as q4build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, MIS, OK = q4.Q4_ERR_INVALID_ARG, q4.Q4_ERR_UNSUPPORTED, q4.Q4_ERR_MISALIGNED, q4.Q4_OK
# disjoint aligned address ranges, 64 MiB apart, never dereferenced
P = [0x100000000 + i * 0x4000000 for i in range(24)]
BIG = 0x2000000
OVL = q4._RunOptions(0x1, 0, 0)
BAD_FLAG = q4._RunOptions(q4.Q4_RUN_EXACT_X, 0, 0)
BAD_RESERVED = q4._RunOptions(0, 1, 0)


@pytest.fixture(scope="module")
def L():
    q4build.build()
    return q4.lib()


def route(L, T=4, E=8, k=2, score=0, opts=None, ws=BIG, **at):
    p = dict(logits=P[0], bias=P[1], mask=P[2], ids=P[3], weights=P[4], offsets=P[5], rows=P[6], pos=P[7], work=P[8])
    p.update(at)
    return L.q4moe_route_run(p["logits"], p["bias"], p["mask"], T, E, k, score, 1, 1.0, p["ids"], p["weights"],
                             p["offsets"], p["rows"], p["pos"], p["work"], ws, opts, None)


def test_route_refusals(L):
    assert route(L, T=-1) == INV and route(L, E=0) == INV and route(L, k=0) == INV and route(L, k=9) == INV
    assert route(L, score=2) == INV
    assert route(L, E=1025) == UNS and route(L, E=64, k=33) == UNS and route(L, T=2 ** 30, E=8, k=4) == UNS
    assert route(L, T=0, logits=None, ids=None) == OK
    for name in ("logits", "ids", "weights", "offsets", "rows", "pos", "work"):
        assert route(L, **{name: None}) == INV, name
    for name in ("logits", "bias", "ids", "weights", "offsets", "rows", "pos", "work"):
        assert route(L, **{name: P[9] + 2}) == MIS, name
    assert route(L, work=P[8] + 128) == MIS
    need = q4.q4moe_route_workspace(5000, 64, 8)
    assert route(L, T=5000, E=64, k=8, ws=need - 1) == INV
    # outputs over inputs, and over one another
    assert route(L, ids=P[0]) == INV and route(L, pos=P[6]) == INV and route(L, work=P[3]) == INV
    assert route(L, opts=ctypes.byref(BAD_FLAG)) == INV and route(L, opts=ctypes.byref(BAD_RESERVED)) == INV


def gemm(L, E=4, R=8, Tx=4, N=64, K=64, g=32, dtype=0, epi=0, opts=None, ws=BIG, **at):
    p = dict(codes=P[0], scales=P[1], zeros=P[2], x=P[3], rows=P[4], offsets=P[5], y=P[6], work=P[7])
    p.update(at)
    return L.q4moe_gemm_run(p["codes"], p["scales"], p["zeros"], p["x"], p["rows"], p["offsets"], p["y"], E, R, Tx, N,
                            K, g, dtype, epi, p["work"], ws, opts, None)


def test_gemm_refusals(L):
    for bad in (dict(R=-1), dict(N=-1), dict(K=0), dict(K=48), dict(g=16), dict(K=96, g=64), dict(E=0), dict(Tx=-1),
                dict(dtype=2), dict(dtype=-1), dict(epi=5), dict(epi=1, N=63), dict(rows=None, Tx=7)):
        assert gemm(L, **bad) == INV, bad
    for bad in (dict(E=1025), dict(R=2 ** 31), dict(Tx=2 ** 31), dict(E=1024, N=2 ** 21), dict(N=2 ** 31)):
        assert gemm(L, **bad) == UNS, bad
    assert gemm(L, R=0, codes=None, x=None) == OK and gemm(L, N=0, codes=None) == OK
    for name in ("codes", "scales", "x", "offsets", "y", "work"):
        assert gemm(L, **{name: None}) == INV, name
    for name, by in (("codes", 8), ("scales", 1), ("x", 8), ("rows", 2), ("offsets", 2), ("y", 2), ("work", 64)):
        assert gemm(L, **{name: P[9] + by}) == MIS, name
    assert gemm(L, dtype=1, y=P[9] + 1) == MIS
    assert gemm(L, ws=q4.q4moe_gemm_workspace(8, 4, 64, 64, 4, q4.Q4_F32) - 1) == INV
    assert gemm(L, y=P[3]) == INV and gemm(L, work=P[6]) == INV and gemm(L, y=P[0]) == INV and gemm(L, y=P[4]) == INV
    assert gemm(L, opts=ctypes.byref(BAD_FLAG)) == INV and gemm(L, opts=ctypes.byref(BAD_RESERVED)) == INV


def norm(L, opts=None, **kw):
    a = dict(T=4, H=64, top_k=2, dtype=0, R=8, y=P[0], pos=P[1], weights=P[2], x=P[3], post_gamma=P[4], gate=P[5],
             gate_stride=0, pre_gamma=P[6], out=P[7], out_norm=P[8], residual_scale=1.0, eps=1e-6)
    a.update(kw)
    return L.q4_block_norm_run(ctypes.byref(q4._BlockNorm(**a)), opts, None)


def test_norm_refusals(L):
    for bad in (dict(T=-1), dict(H=0), dict(top_k=-1), dict(R=-1), dict(dtype=3), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(gate_stride=63), dict(top_k=0), dict(y=None),
                dict(x=None), dict(out=None), dict(pos=None), dict(weights=None), dict(out_norm=None),
                dict(pre_gamma=None)):
        assert norm(L, **bad) == INV, bad
    assert norm(L, H=16385) == UNS and norm(L, top_k=33) == UNS
    assert norm(L, T=0, y=None, x=None, out=None) == OK
    assert L.q4_block_norm_run(None, None, None) == INV
    for name, by in (("y", 8), ("x", 8), ("out", 8), ("out_norm", 4), ("gate", 2), ("post_gamma", 2),
                     ("pre_gamma", 2), ("pos", 2), ("weights", 2)):
        assert norm(L, **{name: P[9] + by}) == MIS, name
    assert norm(L, out=P[0]) == INV and norm(L, out=P[3]) == INV and norm(L, out_norm=P[7]) == INV
    assert norm(L, out=P[5], gate_stride=64) == INV
    assert norm(L, opts=ctypes.byref(BAD_FLAG)) == INV


def block(L, opts=None, **kw):
    a = dict(T=4, E=8, top_k=2, H=64, inner=32, group=32, dtype=1, score=0, renormalize=1, route_scale=1.0,
             residual_scale=1.0, eps=1e-6, up_codes=P[0], up_scales_f16=P[1], up_zeros_u4_or_null=P[2],
             down_codes=P[3], down_scales_f16=P[4], down_zeros_u4_or_null=P[5], logits=P[6], bias_or_null=P[7],
             token_mask_or_null=P[8], a=P[9], x=P[10], post_gamma=P[11], gate=P[12], gate_stride=0, pre_gamma=P[13],
             ids=P[14], route_weights=P[15], out=P[16], out_norm=P[17], workspace=P[18], workspace_bytes=BIG)
    a.update(kw)
    return L.q4moe_block_run(ctypes.byref(q4._MoeBlock(**a)), opts, None)


def test_block_refusals(L):
    for bad in (dict(T=-1), dict(E=0), dict(top_k=9), dict(H=0), dict(inner=0), dict(inner=48), dict(H=48),
                dict(group=16), dict(dtype=2), dict(score=7), dict(eps=-1.0), dict(gate_stride=1),
                dict(out_norm=None), dict(pre_gamma=None), dict(up_codes=None), dict(up_scales_f16=None),
                dict(down_codes=None), dict(down_scales_f16=None), dict(logits=None), dict(a=None), dict(x=None),
                dict(ids=None), dict(route_weights=None), dict(out=None), dict(workspace=None)):
        assert block(L, **bad) == INV, bad
    assert block(L, H=16416) == UNS and block(L, E=2000) == UNS
    assert block(L, T=0, a=None, x=None) == OK
    for name, by in (("up_codes", 8), ("down_codes", 8), ("up_scales_f16", 1), ("a", 8), ("x", 8), ("out", 8),
                     ("out_norm", 8), ("workspace", 128), ("ids", 2), ("logits", 2), ("gate", 1)):
        assert block(L, **{name: P[20] + by}) == MIS, name
    need = q4.q4moe_block_workspace(4, 8, 2, 64, 32, q4.Q4_BF16)
    assert block(L, workspace_bytes=need - 1) == INV
    assert block(L, out=P[10]) == INV and block(L, out=P[9]) == INV and block(L, workspace=P[0]) == INV
    assert L.q4moe_block_run(None, None, None) == INV


def test_workspaces_reject_what_the_calls_reject(L):
    assert L.q4moe_route_workspace(4, 0, 1) == -1 and L.q4moe_route_workspace(4, 2000, 1) == -1
    assert L.q4moe_gemm_workspace(8, 4, 64, 48, 4, 0) == -1 and L.q4moe_gemm_workspace(8, 4, 64, 64, 4, 9) == -1
    assert L.q4moe_block_workspace(4, 8, 2, 64, 48, 0) == -1
    with pytest.raises(q4.Q4Error):
        q4.q4moe_route_workspace(4, 2000, 1)


def test_binding_checks_types_and_shapes():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    i32 = torch.int32
    ids, w, off, rows, pos = z(4, 2, dtype=i32), z(4, 2), z(9, dtype=i32), z(8, dtype=i32), z(4, 2, dtype=i32)
    ws = z(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):
        q4.q4moe_route_run(z(4, 8).double(), ids, w, off, rows, pos, ws, stream=0)
    with pytest.raises(ValueError):
        q4.q4moe_route_run(z(4, 8), ids.long(), w, off, rows, pos, ws, stream=0)
    with pytest.raises(ValueError):
        q4.q4moe_route_run(z(4, 8), ids, w, off[:8], rows, pos, ws, stream=0)
    with pytest.raises(ValueError):   # strided logits
        q4.q4moe_route_run(z(4, 16)[:, ::2], ids, w, off, rows, pos, ws, stream=0)
    codes, scales = z(8, 64, 32, dtype=torch.uint8), z(8, 64, 2).half()
    for x, y in ((z(4, 64).half(), z(8, 64).half()), (z(4, 64), z(8, 64).bfloat16()), (z(4, 32), z(8, 64)),
                 (z(4, 64), z(8, 32))):
        with pytest.raises(ValueError):
            q4.q4moe_gemm_run(codes, scales, None, x, rows, off, y, ws, group=32, stream=0)
    with pytest.raises(ValueError):
        q4.q4_block_norm_run(z(8, 64), z(4, 64), z(4, 64), pos=pos, weights=w, gate=z(4), stream=0)
    with pytest.raises(ValueError):
        q4.q4_block_norm_run(z(8, 64), z(4, 64), z(4, 64).bfloat16(), pos=pos, weights=w, stream=0)


def test_struct_layouts_agree_with_the_header(tmp_path):
    """sizeof and every offset of the two descriptor structs, printed by a C program."""
    lines = []
    for cname, cls in (("q4_block_norm_t", q4._BlockNorm), ("q4moe_block_t", q4._MoeBlock)):
        lines.append(f'printf("%zu\\n", sizeof({cname}));')
        lines += [f'printf("%zu\\n", offsetof({cname}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "q4gemv.h"\nint main(void) {\n' +
                   "\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for cls in (q4._BlockNorm, q4._MoeBlock):
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


# ---------------------------------------------------------------- the reference itself

def test_reference_route_by_hand():
    inf, nan = np.inf, np.nan
    l = np.array([[1.0, 3.0, 3.0, -inf], [nan, -inf, 0.0, -inf], [0.0, 0.0, 0.0, 0.0]], np.float32)
    ids, w, off, rows, pos, _ = ref.route(l, 2, "softmax", True, mask=np.array([1, 1, 0]))
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1]]
    assert w.tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0]]
    assert off.tolist() == [0, 0, 1, 3, 3] and rows.tolist() == [0, 0, 1, -1, -1, -1]
    assert pos.tolist() == [[0, 1], [2, -1], [-1, -1]]


def test_reference_experts_by_hand():
    # one expert, K = 32, codes 9 and zero point 8: every weight is the scale, 0.5
    codes = np.full((1, 2, 16), 0x99, np.uint8)
    W = ref.dequant(codes, np.full((1, 2, 1), 0.5, np.float16), None, 32)
    assert (W == 0.5).all()
    x = np.ones((1, 32), np.float32)
    y, err = ref.experts(W, x, np.array([0, 5], np.int32), np.array([0, 2], np.int32), np.zeros((2, 2)), False, False)
    assert y.tolist() == [[16.0, 16.0], [0.0, 0.0]] and (err >= 0).all()


def test_reference_norm_by_hand():
    y = np.array([[3.0, 4.0], [1.0, 1.0]])
    out, _, a, _ = ref.block_norm(y, np.zeros((1, 2)), np.array([[0, -1]]), np.array([[2.0, 9.0]]), np.ones(2), None,
                                  1.0, np.ones(2), 0.0, 0.0)
    want = np.array([[3.0, 4.0]]) / np.sqrt(12.5)
    assert np.allclose(out, want) and np.allclose(a, want)   # a unit row stays as it is
