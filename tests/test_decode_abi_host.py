"""Host-side checks of the decode operators' C ABI (no GPU needed): every invalid argument is rejected
before any CUDA call, so fake device addresses are never dereferenced."""
import ctypes
import os
import re

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
    text = open(os.path.join(ROOT, "include", "beam_decode.h"), encoding="utf-8").read()
    names = re.findall(r"BEAM_API\s+[\w\s\*]*?\b(beam_\w+)\s*\(", text)
    assert sorted(names) == ["beam_attn_prefix_fwd", "beam_attn_prefix_workspace",
                             "beam_kv_evict_fwd", "beam_w4_matvec_fwd"]
    raw = ctypes.CDLL(rsn.LIB_PATH)
    for nm in names:
        assert hasattr(raw, nm)
        assert nm in rsn.__all__


def attn(lib, out=A, out_stride=6144, lse=A, w_in=None, w_out=None, w_stride=64, q=B, q_stride=6144,
         kc=A, vc=B, slots=1000, dtype=0, ks=1.0, vs=1.0, prefix=A, P=100, table=A, t_stride=64,
         width=64, lens=A, nb=4, q_len=1, nq=48, nkv=8, dim=128, sm=0.1, window=0, ws=A,
         ws_bytes=1 << 40):
    return lib.beam_attn_prefix_fwd(out, out_stride, lse, w_in, w_out, w_stride, q, q_stride, kc,
                                    vc, slots, dtype, ks, vs, prefix, P, table, t_stride, width,
                                    lens, nb, q_len, nq, nkv, dim, sm, window, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dim=64), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(nb=-1), INVALID),
    (dict(q_len=0), INVALID), (dict(nkv=0), INVALID), (dict(nq=50), INVALID),
    (dict(nq=4), INVALID), (dict(nq=1032, nkv=8), INVALID), (dict(P=-1), INVALID),
    (dict(P=1 << 31), INVALID), (dict(width=-1), INVALID), (dict(window=-1), INVALID),
    (dict(slots=-1), INVALID), (dict(slots=1 << 31), INVALID), (dict(sm=NAN), INVALID),
    (dict(sm=INF), INVALID), (dict(dtype=1, ks=0.0), INVALID), (dict(dtype=1, vs=NAN), INVALID),
    (dict(dtype=1, vs=-1.0), INVALID), (dict(out=None), INVALID), (dict(q=None), INVALID),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(prefix=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(ws=None), INVALID),
    (dict(ws_bytes=100), INVALID), (dict(out_stride=6136), INVALID),
    (dict(q_stride=6136), INVALID), (dict(t_stride=63), INVALID), (dict(w_in=A), INVALID),
    (dict(w_out=A, w_stride=63), INVALID), (dict(nb=1 << 26), INVALID),
    (dict(out=A + 8), MISALIGNED), (dict(q=A + 2), MISALIGNED), (dict(kc=A + 8), MISALIGNED),
    (dict(q_stride=6148), MISALIGNED), (dict(table=A + 4), MISALIGNED),
    (dict(prefix=A + 4), MISALIGNED), (dict(lens=A + 2), MISALIGNED), (dict(ws=A + 8), MISALIGNED),
    (dict(w_out=A + 2), MISALIGNED), (dict(lse=A + 2), MISALIGNED),
    (dict(nb=0, out=None, q=None, kc=None, vc=None, lens=None, ws=None, table=None), OK),
])
def test_attention_argument_checks(lib, kw, want):
    assert attn(lib, **kw) == want


def test_attention_workspace(lib):
    f = lib.beam_attn_prefix_workspace
    assert f(-1, 1, 48, 8, 0, 10, 0, 0) == INVALID
    assert f(1, 1, 48, 7, 0, 10, 0, 0) == INVALID
    assert f(0, 1, 48, 8, 0, 10, 0, 0) == 0
    plain, weights = f(8, 1, 48, 8, 100, 5000, 0, 0), f(8, 1, 48, 8, 100, 5000, 0, 1)
    assert 0 < plain < weights
    # exactly enough is enough; one byte less is refused before any launch
    assert attn(lib, nb=8, P=100, width=5000, t_stride=5000, ws_bytes=plain - 1) == INVALID
    with pytest.raises(rsn.BeamError):
        rsn.beam_attn_prefix_workspace(1, 0, 48, 8, 0, 10)


def evict(lib, t_out=A, n_out=A, w_out=A, freed=A, fw=64, t_in=A, n_in=A, w_in=A, rows=4,
          width=128, budget=64, recent=8):
    return lib.beam_kv_evict_fwd(t_out, n_out, w_out, freed, fw, t_in, n_in, w_in, rows, width,
                                 budget, recent, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(width=-1), INVALID), (dict(width=1 << 30, fw=1 << 30), INVALID),
    (dict(budget=-1), INVALID),
    (dict(recent=-1), INVALID), (dict(recent=65), INVALID), (dict(fw=63), INVALID),
    (dict(freed=None), INVALID), (dict(t_out=None), INVALID), (dict(n_out=None), INVALID),
    (dict(w_out=None), INVALID), (dict(t_in=None), INVALID), (dict(n_in=None), INVALID),
    (dict(w_in=None), INVALID), (dict(t_in=A + 4), MISALIGNED), (dict(w_in=A + 2), MISALIGNED),
    (dict(n_in=A + 2), MISALIGNED), (dict(freed=A + 4), MISALIGNED),
    (dict(rows=0, t_out=None, n_out=None, w_out=None, freed=None, t_in=None, n_in=None,
          w_in=None), OK),
])
def test_evict_argument_checks(lib, kw, want):
    assert evict(lib, **kw) == want


def w4(lib, y=A, ys=5120, x=B, xs=6144, w=A, sc=A, z=None, T=4, N=5120, K=6144, group=128):
    return lib.beam_w4_matvec_fwd(y, ys, x, xs, w, sc, z, T, N, K, group, None)


@pytest.mark.parametrize("kw,want", [
    (dict(group=16), UNSUPPORTED), (dict(group=0), UNSUPPORTED), (dict(T=-1), INVALID),
    (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=6144 + 64), INVALID),
    (dict(ys=5119), INVALID), (dict(xs=6136), INVALID), (dict(y=None), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(sc=None), INVALID),
    (dict(x=B + 8), MISALIGNED), (dict(xs=6148), MISALIGNED), (dict(w=A + 8), MISALIGNED),
    (dict(y=A + 1), MISALIGNED), (dict(sc=A + 1), MISALIGNED),
    (dict(T=0, y=None, x=None, w=None, sc=None), OK),
])
def test_w4_argument_checks(lib, kw, want):
    assert w4(lib, **kw) == want


def test_python_refuses_cpu_tensors(lib):
    q = torch.zeros((1, 6, 128), dtype=torch.bfloat16)
    c = torch.zeros((4, 1, 128), dtype=torch.bfloat16)
    i = torch.zeros((1, 4), dtype=torch.int64)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        rsn.beam_attn_prefix_fwd(q, q, c, c, None, i, n, q)
    with pytest.raises(TypeError):
        rsn.beam_kv_evict_fwd(i, n, i, None, i, n, i, 4)
    with pytest.raises(TypeError):
        rsn.beam_w4_matvec_fwd(q[0], q[0], torch.zeros((6, 64), dtype=torch.uint8), q[0])
