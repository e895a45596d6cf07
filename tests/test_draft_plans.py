"""How calls of the draft-checking step's operators are divided (host code, compiled here by itself; no GPU needed)."""
import ctypes
import os
import random
import subprocess

import pytest

import residual_stream_norm_gb300 as rsn

CSRC = os.path.join(os.path.dirname(os.path.abspath(rsn.__file__)), "csrc")
SOURCE = """
#include "draft/draft_plan.h"
extern "C" void plan(int B, int q_len, int n_q, int n_kv, int64_t width, int64_t window, int64_t n_sink, int group,
                     int64_t *to)
{
    const beam::Kv4AttnPlan p = beam::kv4_attn_plan(B, q_len, n_q, n_kv, width, window, n_sink, group);
    const int64_t all[] = {p.heads, p.R, p.nt, p.rtiles, p.teams, p.ctas, p.warps, p.gang, p.bytes,
                           beam::kv4::warps_of(p.nt, 128 / group)};
    for (int64_t x : all)
        *to++ = x;
}
extern "C" int ranks(int64_t B, int64_t V) { return beam::verify_ranks(B, V); }
"""
NAMES = ("heads", "R", "nt", "rtiles", "teams", "ctas", "warps", "gang", "bytes", "fit")


@pytest.fixture(scope="module")
def so(tmp_path_factory):
    d = tmp_path_factory.mktemp("plans")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror", f"-I{CSRC}", "-o", str(d / "plan.so"),
                    str(d / "plan.cpp")], check=True)
    so = ctypes.CDLL(str(d / "plan.so"))
    so.plan.argtypes = [ctypes.c_int] * 4 + [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.c_void_p]
    so.plan.restype = None
    so.ranks.argtypes = [ctypes.c_int64] * 2
    return so


def plan(so, B, q_len=1, n_q=48, n_kv=8, width=1000, window=0, n_sink=0, group=128):
    to = (ctypes.c_int64 * len(NAMES))()
    so.plan(B, q_len, n_q, n_kv, width, window, n_sink, group, to)
    return dict(zip(NAMES, to))


def test_attention_plans_hold_together(so):
    rng = random.Random(0)
    for _ in range(3000):
        n_kv = rng.choice([1, 2, 5, 8, 64])
        n_q, B, q_len = n_kv * rng.choice([1, 2, 6, 16]), rng.choice([1, 2, 19, 150, 700, 5000]), rng.choice([1, 2, 5, 64])
        width = int(2 ** rng.uniform(0, 18))
        args = dict(B=B, q_len=q_len, n_q=n_q, n_kv=n_kv, width=width, window=rng.choice([0, 0, 1, 512, 3000]),
                    n_sink=rng.choice([0, 4, 100]), group=rng.choice([32, 64, 128]))
        p = plan(so, **args)
        assert p["nt"] * 8 * p["rtiles"] >= p["R"] and 1 <= p["nt"] <= 3, args
        assert 1 <= p["warps"] <= p["fit"] and p["ctas"] >= 1, args
        if p["gang"]:
            assert p["warps"] % p["gang"] == 0, args
        else:  # every team's warps have a place, and the warps that count the tiles are there
            assert p["warps"] >= 8 and (p["ctas"] == 152 or p["ctas"] * p["warps"] >= p["teams"] * n_kv * p["rtiles"])
        assert p["bytes"] == p["teams"] * n_kv * p["rtiles"] * 2 * p["nt"] * 8 * 130 * 4, args


@pytest.mark.parametrize("group", [32, 64, 128])
def test_one_long_sequence_is_shared_out(so, group):
    # however evenly the units divide over the SMs: a unit that its gang alone would take for long is cut
    for n_kv, n_q in ((1, 6), (2, 12), (8, 48), (8, 8)):
        for B in (1, 2, 8, 16, 17, 18, 19, 37, 38, 57, 76, 95, 114, 128, 150, 152, 190, 304, 700):
            for q_len in (1, 2, 4):
                for width in (5000, 8100, 12_160, 24_320, 100_000, 1 << 20):
                    p = plan(so, B=B, q_len=q_len, n_q=n_q, n_kv=n_kv, width=width, group=group)
                    assert p["gang"] == 0, (B, q_len, n_q, width)
                p = plan(so, B=B, q_len=q_len, n_q=n_q, n_kv=n_kv, width=100_000, window=8000, group=group)
                assert p["gang"] == 0


def test_short_sequences_are_taken_whole(so):
    for B, q_len, width, window in ((1, 1, 500, 0), (8, 1, 2000, 0), (19, 1, 4000, 0), (19, 4, 2000, 0), (128, 1, 500, 0),
                                    (1000, 1, 200, 0), (128, 1, 8192, 512), (50, 1, 8192, 512), (300, 1, 8192, 1024),
                                    (128, 4, 8192, 1024)):
        assert plan(so, B=B, q_len=q_len, width=width, window=window)["gang"] > 0, (B, q_len, width, window)


def test_verification_takes_no_more_blocks_than_a_vocabulary_has_work_for(so):
    for V in (1, 500, 2047, 2048, 8192, 160_000, (1 << 20) - 1):
        for B in (1, 16, 76, 77, 152, 153, 400, 5000):
            r = so.ranks(B, V)
            assert r in (1, 2, 4, 8) and (r == 1 or V >= r * 8 * 128)


def test_verification_of_the_most_sequences_fits_a_grid(so):
    # sequences may share their distributions (strides of 0), so there may be as many as the check lets through
    for V in (1, 2048, 9000, 64_000, (1 << 20) - 1):
        for B in ((1 << 28) + 1, 1 << 29, (1 << 30) + 152, (1 << 31) - 1):
            assert B * so.ranks(B, V) <= (1 << 31) - 1, (B, V)
