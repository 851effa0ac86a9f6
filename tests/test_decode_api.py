"""Host-side checks of the calls for several continuations of one prompt: workspaces, refusals,
struct layouts, rotary frequencies.

Every call below fails a check that runs before the first CUDA call, or is an empty problem, so
no pointer here is ever dereferenced."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import gemm_decode_gb300 as q4
from gemm_decode_gb300 import build as q4build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, MIS, OK = q4.Q4_ERR_INVALID_ARG, q4.Q4_ERR_UNSUPPORTED, q4.Q4_ERR_MISALIGNED, q4.Q4_OK
# disjoint aligned address ranges, 64 MiB apart, never dereferenced
P = [0x100000000 + i * 0x4000000 for i in range(24)]
BIG = 0x2000000
BAD_FLAG = q4._RunOptions(q4.Q4_RUN_EXACT_X, 0, 0)
BAD_RESERVED = q4._RunOptions(0, 1, 0)


@pytest.fixture(scope="module")
def L():
    q4build.build()
    return q4.lib()


def cache(**kw):
    a = dict(k=P[0], v=P[1], dtype=q4.Q4_BF16, heads=2, D=64, page=16, pages=10, page_stride=2048, head_stride=1024,
             row_stride=64)
    a.update(kw)
    return q4._KvCache(**a)


BAD_CACHES = (dict(dtype=0), dict(dtype=3), dict(heads=0), dict(D=0), dict(page=0), dict(pages=-1),
              dict(page_stride=2047), dict(head_stride=1023), dict(row_stride=63), dict(page_stride=-2048),
              dict(row_stride=-64), dict(head_stride=0), dict(page_stride=2 ** 50))


def rope(L, opts=None, c=None, **kw):
    a = dict(T=3, Hq=4, dtype=0, rot=64, layout=0, scale=1.0, eps=1e-6, q=P[2], k=P[3], v=P[4], q_stride=256,
             k_stride=128, v_stride=128, q_gamma=P[5], k_gamma=P[6], positions=P[7], inv_freq=P[8], slots=P[9],
             q_out=P[10], cache=c or cache())
    a.update(kw)
    return L.q4_rope_append_run(ctypes.byref(q4._RopeAppend(**a)), opts, None)


def test_rope_refusals(L):
    for bad in (dict(T=-1), dict(Hq=0), dict(dtype=2), dict(dtype=-1), dict(rot=-2), dict(rot=3), dict(rot=66),
                dict(layout=2), dict(scale=math.nan), dict(scale=math.inf), dict(eps=-1.0), dict(eps=math.nan),
                dict(q_stride=255), dict(k_stride=127), dict(v_stride=127), dict(q_stride=-256), dict(q=None),
                dict(q_out=None), dict(positions=None), dict(inv_freq=None), dict(k=None), dict(v=None),
                dict(q_out=P[2]), dict(q_out=P[0]), dict(q_out=P[1]), dict(q_out=P[9]), dict(k=P[0]), dict(v=P[1]),
                dict(q=P[1]), dict(slots=P[0])):
        assert rope(L, **bad) == INV, bad
    for bad in BAD_CACHES + (dict(k=None), dict(v=None), dict(v=P[0])):
        assert rope(L, c=cache(**bad)) == INV, bad
    wide = dict(D=258, page_stride=10000, head_stride=5000, row_stride=258)
    assert rope(L, c=cache(**wide), rot=0, q_stride=2000, k_stride=2000, v_stride=2000) == UNS
    assert rope(L, Hq=2 ** 20, q_stride=2 ** 30) == UNS
    for name, by in (("q", 2), ("k", 2), ("v", 2), ("q_out", 1), ("q_gamma", 2), ("k_gamma", 2), ("positions", 2),
                     ("inv_freq", 2), ("slots", 2)):
        assert rope(L, **{name: P[11] + by}) == MIS, name
    assert rope(L, dtype=1, q=P[11] + 1) == MIS and rope(L, c=cache(k=P[11] + 1)) == MIS
    assert rope(L, T=0, q=None, q_out=None) == OK
    assert L.q4_rope_append_run(None, None, None) == INV
    assert rope(L, opts=ctypes.byref(BAD_FLAG)) == INV and rope(L, opts=ctypes.byref(BAD_RESERVED)) == INV


def test_rope_frequencies():
    f = q4.q4_rope_frequencies(64, 10000.0).numpy()
    want = 10000.0 ** (-np.arange(0, 64, 2) / 64.0)
    assert np.array_equal(f, want.astype(np.float32))
    assert np.array_equal(q4.q4_rope_frequencies(64, 10000.0, q4.Q4_ROPE_LINEAR, 4.0).numpy(),
                          (want / 4).astype(np.float32))
    b = q4.q4_rope_frequencies(128, 500000.0, q4.Q4_ROPE_BANDS, 8.0, 8192, 1.0, 4.0).numpy().astype(np.float64)
    plain = 500000.0 ** (-np.arange(0, 128, 2) / 128.0)
    turns = 8192 * plain / (2 * np.pi)
    assert np.allclose(b[turns >= 4], plain[turns >= 4], rtol=2.0 ** -23) and (turns >= 4).any()
    assert np.allclose(b[turns <= 1], plain[turns <= 1] / 8, rtol=2.0 ** -23) and (turns <= 1).any()
    mid = (turns > 1) & (turns < 4)
    keep = (turns[mid] - 1) / 3
    assert mid.any() and np.allclose(b[mid], plain[mid] * (keep + (1 - keep) / 8), rtol=2.0 ** -22)
    assert q4.q4_rope_frequencies(0).numel() == 0
    for bad in (dict(rot=-2), dict(rot=5), dict(base=0.0), dict(base=math.nan), dict(kind=3), dict(kind=1, factor=0.5),
                dict(kind=2, factor=math.inf, trained=1.0), dict(kind=2, factor=2.0), dict(kind=2, trained=9.0, low=4.0)):
        a = dict(rot=8)
        a.update(bad)
        with pytest.raises(q4.Q4Error):
            q4.q4_rope_frequencies(**a)


def attn(L, opts=None, c=None, **kw):
    a = dict(S=5, Hq=4, groups=2, out_dtype=q4.Q4_BF16, max_shared_pages=3, max_own_pages=2, scale=0.1, q=P[2],
             q_stride=256, cache=c or cache(), group_offsets=P[3], shared_pages=P[4], shared_lens=P[5], limits=P[6],
             own_pages=P[7], own_lens=P[8], out=P[9], lse=P[10], workspace=P[11], workspace_bytes=BIG)
    a.update(kw)
    return L.q4_prefix_attn_run(ctypes.byref(q4._PrefixAttn(**a)), opts, None)


def test_attention_refusals(L):
    for bad in (dict(S=-1), dict(Hq=0), dict(Hq=3), dict(groups=-1), dict(out_dtype=q4.Q4_F16), dict(out_dtype=3),
                dict(max_shared_pages=-1), dict(max_own_pages=-1), dict(scale=math.nan), dict(scale=math.inf),
                dict(q_stride=248), dict(q_stride=-256), dict(q=None), dict(out=None), dict(workspace=None),
                dict(shared_lens=None), dict(shared_pages=None), dict(group_offsets=None), dict(own_lens=None),
                dict(own_pages=None), dict(groups=0, own_pages=None, own_lens=None), dict(out=P[2]), dict(out=P[0]),
                dict(out=P[1]), dict(lse=P[9]), dict(workspace=P[9]), dict(lse=P[4]), dict(workspace=P[7]),
                dict(out=P[6])):
        assert attn(L, **bad) == INV, bad
    for bad in BAD_CACHES + (dict(k=None), dict(v=None), dict(pages=0)):
        assert attn(L, c=cache(**bad)) == INV, bad
    for c in (dict(D=96, row_stride=96, head_stride=2000, page_stride=4000), dict(page=8), dict(page=24, head_stride=2000, page_stride=4000)):
        assert attn(L, c=cache(**c), q_stride=4096) == UNS, c
    for bad in (dict(groups=6), dict(S=2 ** 20 + 1), dict(Hq=258), dict(max_shared_pages=2 ** 27),
                dict(max_own_pages=2 ** 27), dict(S=2 ** 20, Hq=4096)):
        assert attn(L, **bad) == UNS, bad
    need = q4.q4_prefix_attn_workspace(5, 2, 4, 2, 64)
    assert attn(L, workspace_bytes=need - 1) == INV
    for name, by in (("q", 8), ("out", 8), ("workspace", 128), ("lse", 2), ("group_offsets", 2), ("shared_pages", 2),
                     ("shared_lens", 2), ("limits", 2), ("own_pages", 2), ("own_lens", 2)):
        assert attn(L, **{name: P[12] + by}) == MIS, name
    assert attn(L, q_stride=260) == MIS and attn(L, c=cache(k=P[12] + 8)) == MIS
    assert attn(L, c=cache(row_stride=68, head_stride=2048, page_stride=4096)) == MIS
    assert attn(L, S=0, groups=0, q=None, out=None) == OK
    assert L.q4_prefix_attn_run(None, None, None) == INV
    assert attn(L, opts=ctypes.byref(BAD_FLAG)) == INV and attn(L, opts=ctypes.byref(BAD_RESERVED)) == INV
    for bad in ((-1, 0, 4, 2, 64), (4, 5, 4, 2, 64), (4, 1, 3, 2, 64), (4, 1, 4, 2, 80), (4, 1, 0, 1, 64)):
        with pytest.raises(q4.Q4Error):
            q4.q4_prefix_attn_workspace(*bad)


def beam(L, groups=2, W=3, K=4, V=100, eos=7, opts=None, ws=BIG, stride=100, **at):
    p = dict(logits=P[0], scores=P[1], finished=P[2], tokens=P[3], parents=P[4], out=P[5], fin=P[6], work=P[7])
    p.update(at)
    return L.q4_beam_step_run(p["logits"], stride, p["scores"], p["finished"], groups, W, K, V, eos, p["tokens"],
                              p["parents"], p["out"], p["fin"], p["work"], ws, opts, None)


def test_beam_refusals(L):
    for bad in (dict(groups=-1), dict(W=0), dict(K=0), dict(V=0), dict(eos=-2), dict(eos=100), dict(eos=-1),
                dict(stride=99), dict(stride=-100), dict(logits=None), dict(scores=None), dict(tokens=None),
                dict(parents=None), dict(out=None), dict(work=None), dict(tokens=P[0]), dict(parents=P[3]),
                dict(out=P[1]), dict(fin=P[2]), dict(work=P[0])):
        assert beam(L, **bad) == INV, bad
    for bad in (dict(W=33), dict(K=33), dict(V=2 ** 31 - 1, stride=2 ** 31, eos=-1), dict(groups=2 ** 30)):
        assert beam(L, **bad) == UNS, bad
    assert beam(L, ws=q4.q4_beam_step_workspace(2, 3, 4, 100) - 1) == INV
    for name in ("logits", "scores", "tokens", "parents", "out"):
        assert beam(L, **{name: P[8] + 2}) == MIS, name
    assert beam(L, work=P[8] + 128) == MIS
    assert beam(L, groups=0, logits=None, scores=None) == OK
    assert beam(L, opts=ctypes.byref(BAD_FLAG)) == INV and beam(L, opts=ctypes.byref(BAD_RESERVED)) == INV
    with pytest.raises(q4.Q4Error):
        q4.q4_beam_step_workspace(1, 33, 1, 10)


def reorder(L, opts=None, **kw):
    a = dict(groups=2, W=3, max_pages=5, planes=4, heads=2, page=16, pages=20, row_bytes=128, plane_stride=128 * 640,
             page_stride=128 * 32, head_stride=128 * 16, row_stride=128, pool=P[0], tables=P[1], lens=P[2],
             parents=P[3], spare=P[4], out_tables=P[5], out_spare=P[6])
    a.update(kw)
    return L.q4_beam_reorder_run(ctypes.byref(q4._BeamReorder(**a)), opts, None)


def test_reorder_refusals(L):
    for bad in (dict(groups=-1), dict(W=0), dict(max_pages=-1), dict(planes=-1), dict(heads=0), dict(page=0),
                dict(pages=-1), dict(row_bytes=0), dict(row_bytes=127), dict(row_stride=126), dict(head_stride=1000),
                dict(page_stride=128 * 31), dict(plane_stride=128 * 639), dict(page_stride=-2), dict(pool=None),
                dict(tables=None), dict(lens=None), dict(parents=None), dict(spare=None), dict(out_tables=None),
                dict(out_spare=None), dict(out_tables=P[1]), dict(out_spare=P[4]), dict(pool=P[1]), dict(out_spare=P[5])):
        assert reorder(L, **bad) == INV, bad
    for bad in (dict(W=1025), dict(groups=2 ** 30), dict(pages=2 ** 31), dict(heads=2 ** 20, page=2 ** 10)):
        assert reorder(L, **bad) == UNS, bad
    for name in ("tables", "lens", "parents", "spare", "out_tables", "out_spare"):
        assert reorder(L, **{name: P[8] + 2}) == MIS, name
    assert reorder(L, pool=P[8] + 1) == MIS and reorder(L, row_stride=129, head_stride=4096, page_stride=8192,
                                                         plane_stride=8192 * 20) == MIS
    assert reorder(L, groups=0, pool=None, tables=None) == OK
    assert L.q4_beam_reorder_run(None, None, None) == INV
    assert reorder(L, opts=ctypes.byref(BAD_FLAG)) == INV


def test_struct_layouts_match_the_header(tmp_path):
    structs = {"q4_kv_cache_t": q4._KvCache, "q4_rope_append_t": q4._RopeAppend, "q4_prefix_attn_t": q4._PrefixAttn,
               "q4_beam_reorder_t": q4._BeamReorder}
    src = tmp_path / "s.c"
    lines = ['#include "q4gemv.h"', "#include <stddef.h>", "#include <stdio.h>", "int main(void) {"]
    for name, s in structs.items():
        lines.append(f'printf("{name} %zu", sizeof({name}));')
        lines += [f'printf(" %zu", offsetof({name}, {f[0]}));' for f in s._fields_]
        lines.append('printf("\\n");')
    src.write_text("\n".join(lines) + "return 0; }\n")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    for line, (name, s) in zip(out.splitlines(), structs.items()):
        want = [ctypes.sizeof(s)] + [getattr(s, f[0]).offset for f in s._fields_]
        assert line.split() == [name] + [str(v) for v in want]


def test_packed_structures_match_the_layouts():
    """The binding packs the structures as bytes: sizes and places of the fields."""
    for packer, s in ((q4._ROPE, q4._RopeAppend), (q4._ATTN, q4._PrefixAttn), (q4._REORDER, q4._BeamReorder)):
        assert packer.size == ctypes.sizeof(s)
        flat = []
        for name, kind in s._fields_:
            flat += [(name, f) for f, _ in kind._fields_] if hasattr(kind, "_fields_") else [(name, None)]
        a = s.from_buffer_copy(packer.pack(*range(1, len(flat) + 1)))
        for i, (name, inner) in enumerate(flat):
            have = getattr(a, name) if inner is None else getattr(getattr(a, name), inner)
            assert have == i + 1, (name, inner)


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    import torch
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError):
        q4.q4_rope_append_run(x, None, None, torch.zeros(2, dtype=torch.int32), torch.zeros(32), x.bfloat16(), None, None)
    with pytest.raises(ValueError):
        q4.q4_prefix_attn_run(x.bfloat16(), x, x, x, x)
    with pytest.raises(ValueError):
        q4.q4_beam_step_run(torch.zeros(2, 9), torch.zeros(1, 2), None, None, None, None)
    with pytest.raises(ValueError):
        q4.q4_beam_reorder_run(None, None, None, None, None, None, torch.zeros(1, 1, 1, 1, 2))


def test_strides_whose_products_pass_64_bits_are_refused(L):
    most = 2 ** 31 - 1
    for name in ("q_stride", "k_stride", "v_stride"):
        assert rope(L, T=most, **{name: 2 ** 43}) == UNS, name
    assert attn(L, S=2 ** 20, q_stride=2 ** 43) == UNS
    assert beam(L, groups=2 ** 26, W=32, stride=2 ** 43) == UNS
    for c in (cache(pages=2 ** 60), cache(pages=2 ** 31 - 1, page_stride=2 ** 43)):
        assert rope(L, c=c) == UNS and attn(L, c=c) == UNS
