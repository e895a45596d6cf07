"""Host-side checks of the C ABI of the draft-checking step's operators (no GPU needed): every invalid
argument is rejected before any CUDA call, so fake device addresses are never dereferenced."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import residual_stream_norm_gb300 as rsn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, MISALIGNED, UNSUPPORTED = 0, -1, -2, -3
A, B = 0x10000, 0x20000
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    rsn.build()
    return rsn.lib()


def test_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "beam_draft.h"), encoding="utf-8").read()
    names = re.findall(r"BEAM_API\s+[\w\s\*]*?\b(beam_\w+)\s*\(", text)
    assert sorted(names) == ["beam_attn_kv4_fwd", "beam_attn_kv4_workspace", "beam_draft_verify_fwd",
                             "beam_kv4_write_fwd", "beam_moe_layer_fwd", "beam_moe_layer_workspace"]
    raw = ctypes.CDLL(rsn.LIB_PATH)
    for nm in names:
        assert hasattr(raw, nm)
        assert nm in rsn.__all__


def write(lib, kc=A, vc=A, ks=A, vs=A, slots=100, group=128, k=A, k_stride=1024, v=A, v_stride=1024, slot=A,
          T=4, n_kv=8, dim=128):
    return lib.beam_kv4_write_fwd(kc, vc, ks, vs, slots, group, k, k_stride, v, v_stride, slot, T, n_kv, dim,
                                  None)


@pytest.mark.parametrize("kw,want", [
    (dict(dim=64), UNSUPPORTED), (dict(group=16), UNSUPPORTED), (dict(group=0), UNSUPPORTED),
    (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(n_kv=0), INVALID), (dict(n_kv=1025), INVALID),
    (dict(slots=-1), INVALID), (dict(slots=1 << 31), INVALID), (dict(kc=None), INVALID),
    (dict(vc=None), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(slot=None), INVALID), (dict(k_stride=1016), INVALID),
    (dict(v_stride=1016), INVALID), (dict(kc=A + 8), MISALIGNED), (dict(vc=A + 4), MISALIGNED),
    (dict(ks=A + 2), MISALIGNED), (dict(vs=A + 4, group=64), MISALIGNED),
    (dict(ks=A + 8, group=32), MISALIGNED), (dict(k=A + 8), MISALIGNED), (dict(k_stride=1028), MISALIGNED),
    (dict(v_stride=1026), MISALIGNED), (dict(slot=A + 4), MISALIGNED),
    (dict(T=0, kc=None, vc=None, ks=None, vs=None, k=None, v=None, slot=None), OK),
    (dict(slots=0, kc=None, vc=None, ks=None, vs=None), OK),
])
def test_write_argument_checks(lib, kw, want):
    assert write(lib, **kw) == want


def attn(lib, out=A, out_stride=6144, lse=A, q=B, q_stride=6144, kc=A, vc=B, ks=A, vs=B, slots=1000,
         group=128, table=A, t_stride=64, width=64, lens=A, nb=4, q_len=1, nq=48, nkv=8, dim=128, sm=0.1,
         window=0, n_sink=0, ws=A, ws_bytes=1 << 40):
    return lib.beam_attn_kv4_fwd(out, out_stride, lse, q, q_stride, kc, vc, ks, vs, slots, group, table,
                                 t_stride, width, lens, nb, q_len, nq, nkv, dim, sm, window, n_sink, ws,
                                 ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dim=64), UNSUPPORTED), (dict(group=256), UNSUPPORTED), (dict(nb=-1), INVALID),
    (dict(q_len=0), INVALID), (dict(nkv=0), INVALID), (dict(nq=50), INVALID), (dict(nq=4), INVALID),
    (dict(nq=1032, nkv=8), INVALID), (dict(width=-1), INVALID), (dict(width=1 << 30), INVALID),
    (dict(window=-1), INVALID), (dict(n_sink=-1), INVALID), (dict(slots=-1), INVALID),
    (dict(slots=1 << 31), INVALID), (dict(sm=NAN), INVALID), (dict(sm=INF), INVALID),
    (dict(nb=1 << 26), INVALID), (dict(nb=1 << 30, q_len=1 << 30), INVALID), (dict(out=None), INVALID),
    (dict(q=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(ks=None), INVALID),
    (dict(vs=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=100), INVALID), (dict(out_stride=6136), INVALID),
    (dict(q_stride=6136), INVALID), (dict(t_stride=63), INVALID), (dict(out=A + 8), MISALIGNED),
    (dict(q=A + 2), MISALIGNED), (dict(kc=A + 8), MISALIGNED), (dict(ks=A + 2), MISALIGNED),
    (dict(vs=A + 4, group=64), MISALIGNED), (dict(vs=A + 8, group=32), MISALIGNED),
    (dict(q_stride=6148), MISALIGNED), (dict(out_stride=6148), MISALIGNED), (dict(table=A + 4), MISALIGNED),
    (dict(lens=A + 2), MISALIGNED), (dict(lse=A + 2), MISALIGNED), (dict(ws=A + 8), MISALIGNED),
    (dict(nb=0, out=None, q=None, kc=None, vc=None, lens=None, ws=None, table=None), OK),
])
def test_attention_argument_checks(lib, kw, want):
    assert attn(lib, **kw) == want


def test_attention_workspace(lib):
    f = lib.beam_attn_kv4_workspace
    assert f(-1, 1, 48, 8, 10, 0, 0) == INVALID
    assert f(1, 1, 48, 7, 10, 0, 0) == INVALID
    assert f(0, 1, 48, 8, 10, 0, 0) == 0
    n = f(8, 1, 48, 8, 5000, 0, 0)
    assert n > 0 and attn(lib, nb=8, width=5000, t_stride=5000, ws_bytes=n - 1) == INVALID
    # any window from the table's width on is none, and any number of sinks all keys
    most = (1 << 63) - 1
    for window, n_sink in ((most, 0), (most, most), (3, most), (5000, 4)):
        assert f(8, 1, 48, 8, 5000, window, n_sink) == n
    with pytest.raises(rsn.BeamError):
        rsn.beam_attn_kv4_workspace(1, 0, 48, 8, 10)


PLANS = """
import sys
import residual_stream_norm_gb300 as rsn
lib = rsn.lib()
f = lib.beam_attn_kv4_workspace
# no sequences: any number of query rows, with and without a launch to plan
for q_len, n_q in ((4194304, 1024), (2147483647, 1024), (1 << 30, 1)):
    assert f(0, q_len, n_q, 1, 100, 0, 0) == 0
    assert lib.beam_attn_kv4_fwd(None, 0, None, None, 0, None, None, None, None, 0, 128, None, 0, 100, None, 0,
                                 q_len, n_q, 1, 128, 0.1, 0, 0, None, 0, None) == 0
# the most query rows: parts of 24 rows, 130 floats a row, two a unit
rows = 2147483647
assert f(1, rows, 1, 1, 100, 0, 0) == -(-rows // 24) * 2 * 24 * 130 * 4
assert f(1, rows - 7, 1, 1, 100, 0, 0) == -(-(rows - 7) // 24) * 2 * 24 * 130 * 4
assert f(2, rows, 1, 1, 100, 0, 0) == -1 and f(1, 1 << 21, 1024, 1, 100, 0, 0) == -1
"""


def test_attention_plans_of_the_most_query_rows(lib):
    # in a process of its own, which a division by a row count that wrapped to zero would end
    r = subprocess.run([sys.executable, "-c", PLANS], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])


def moe(lib, out=A, out_stride=512, ids=A, w=A, x=A, x_stride=512, rw=A, rb=A, w13=A, w2=A, first=0,
        local=256, scaling=2.5, T=4, H=512, F=64, ws=A, ws_bytes=1 << 40):
    return lib.beam_moe_layer_fwd(out, out_stride, ids, w, x, x_stride, rw, rb, w13, w2, first, local, scaling,
                                  T, H, F, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=257), UNSUPPORTED), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=516), INVALID),
    (dict(H=16392, out_stride=16392, x_stride=16392), INVALID), (dict(F=4), INVALID), (dict(F=60), INVALID),
    (dict(F=32776), INVALID), (dict(local=0), INVALID), (dict(local=257), INVALID), (dict(first=-1), INVALID),
    (dict(first=1), INVALID), (dict(first=225, local=32), INVALID), (dict(scaling=NAN), INVALID),
    (dict(scaling=INF), INVALID), (dict(out=None), INVALID), (dict(x=None), INVALID), (dict(rw=None), INVALID),
    (dict(rb=None), INVALID), (dict(w13=None), INVALID), (dict(w2=None), INVALID), (dict(ws=None), INVALID),
    (dict(out_stride=504), INVALID), (dict(x_stride=504), INVALID), (dict(out=A + 8), MISALIGNED),
    (dict(x=A + 8), MISALIGNED), (dict(x_stride=516), MISALIGNED), (dict(out_stride=514), MISALIGNED),
    (dict(rw=A + 4), MISALIGNED), (dict(rb=A + 4), MISALIGNED), (dict(w13=A + 8), MISALIGNED),
    (dict(w2=A + 8), MISALIGNED), (dict(ids=A + 2), MISALIGNED), (dict(w=A + 2), MISALIGNED),
    (dict(ws=A + 8), MISALIGNED),
    (dict(T=0, out=None, x=None, rw=None, rb=None, w13=None, w2=None, ws=None), OK),
])
def test_moe_argument_checks(lib, kw, want):
    assert moe(lib, **kw) == want


def test_moe_workspace(lib):
    f = lib.beam_moe_layer_workspace
    assert f(0, 512, 64, 256) == 0 and f(4, 512, 60, 256) == INVALID and f(257, 512, 64, 256) == UNSUPPORTED
    n = f(4, 512, 64, 256)
    assert n > 0 and moe(lib, ws_bytes=n - 1) == INVALID
    with pytest.raises(rsn.BeamError):
        rsn.beam_moe_layer_workspace(-1, 512, 64)


def verify(lib, out=A, acc=A, tokens=A, lens=None, target=A, t_seq=500, t_pos=100, draft=A, d_seq=400,
           d_pos=100, dtype=0, ua=A, us=A, nb=2, k=4, V=100):
    return lib.beam_draft_verify_fwd(out, acc, tokens, lens, target, t_seq, t_pos, draft, d_seq, d_pos, dtype,
                                     ua, us, nb, k, V, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(nb=-1), INVALID),
    (dict(nb=1 << 31), INVALID), (dict(k=-1), INVALID), (dict(k=1025), INVALID), (dict(V=0), INVALID),
    (dict(V=1 << 20), INVALID), (dict(t_seq=-1), INVALID), (dict(t_pos=-1), INVALID), (dict(d_seq=-1), INVALID),
    (dict(d_pos=-1), INVALID), (dict(out=None), INVALID), (dict(acc=None), INVALID), (dict(tokens=None), INVALID),
    (dict(target=None), INVALID), (dict(ua=None), INVALID), (dict(us=None), INVALID),
    (dict(out=A + 4), MISALIGNED), (dict(acc=A + 2), MISALIGNED), (dict(tokens=A + 4), MISALIGNED),
    (dict(lens=A + 2), MISALIGNED), (dict(target=A + 2), MISALIGNED), (dict(draft=A + 2), MISALIGNED),
    (dict(target=A + 1, dtype=1), MISALIGNED), (dict(ua=A + 2), MISALIGNED), (dict(us=A + 1), MISALIGNED),
    (dict(nb=0, out=None, acc=None, tokens=None, target=None, draft=None, ua=None, us=None), OK),
])
def test_verify_argument_checks(lib, kw, want):
    assert verify(lib, **kw) == want


def test_python_refuses_what_does_not_fit(lib):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    i64, f32 = torch.zeros((1, 4), dtype=torch.int64), torch.zeros((1, 4))
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        rsn.beam_kv4_write_fwd(u8(4, 1, 64), u8(4, 1, 64), bf(4, 1, 1, 2), bf(4, 1, 1, 2), bf(4, 1, 128),
                               bf(4, 1, 128), i64[0])
    with pytest.raises(TypeError):
        rsn.beam_attn_kv4_fwd(bf(1, 6, 128), bf(1, 6, 128), u8(4, 1, 64), u8(4, 1, 64), bf(4, 1, 1, 2),
                              bf(4, 1, 1, 2), i64, n, u8(100))
    with pytest.raises(TypeError):
        rsn.beam_moe_layer_fwd(bf(4, 64), bf(4, 64), torch.zeros(256, 64), torch.zeros(256), bf(256, 32, 64),
                               bf(256, 64, 16), u8(100))
    with pytest.raises(TypeError):
        rsn.beam_draft_verify_fwd(i64, n, i64[:, :3], torch.zeros(1, 4, 9), None, f32[:, :3], f32[0, :1])


@pytest.mark.parametrize("bad", [1 << 32, (1 << 32) + 1, -(1 << 32) + 1, (1 << 64) + 1])
def test_sizes_that_the_c_types_cannot_hold(lib, bad):
    # ctypes would cut them off to 0 or 1
    for i in range(4):
        sizes = [1, 1, 8, 8, 10]
        sizes[i] = bad
        with pytest.raises(rsn.BeamError):
            rsn.beam_attn_kv4_workspace(*sizes)
    for kw in (dict(window=(1 << 64) + 5), dict(n_sink=1 << 64), dict(table_width=(1 << 64) + 3)):
        with pytest.raises(rsn.BeamError):
            rsn.beam_attn_kv4_workspace(**{**dict(B=1, q_len=1, n_q_heads=8, n_kv_heads=8, table_width=10), **kw})
    for i in range(1, 4):
        sizes = [4, 64, 16, 256]
        sizes[i] = bad * 8
        with pytest.raises(rsn.BeamError):
            rsn.beam_moe_layer_workspace(*sizes)
