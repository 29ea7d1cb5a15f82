"""Host logic of the transformer operators' choice of kernel, tile and split
(choose_attention, choose_linear), no GPU: a small C++ probe links libcc3d.so
and reports what a call takes.  The GPU tests' cases have to reach every
kernel, so that a change of the measured constants cannot leave one untested;
every choice has to cover the call's rows; and the choices that the timed
cases rest on are pinned."""
import os
import random
import shutil
import subprocess

import pytest

from tests.test_gpu_attention import KERNELS, LONG_FRAMES
from tests.test_gpu_linear import CHOICES
from tests.test_gpu_ops_failure import PAIRS, SPLITS
from video_vae_causal_implicit_b200 import build as cbuild
from video_vae_causal_implicit_b200 import cc3d

HERE = os.path.dirname(os.path.abspath(__file__))
CUDA = os.environ.get("CUDA_HOME") or "/usr/local/cuda"


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    inc = os.path.join(CUDA, "include")
    if shutil.which("g++") is None or not os.path.exists(os.path.join(inc, "cuda.h")):
        pytest.skip("needs g++ and the CUDA headers")
    cbuild.build()
    exe = str(tmp_path_factory.mktemp("ops") / "ops_probe")
    libdir = os.path.dirname(cc3d.LIB_PATH)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", cbuild.CSRC, "-I", cbuild.INCLUDE, "-I", inc,
                    os.path.join(HERE, "plan", "ops_probe.cpp"), "-o", exe, "-L", libdir, "-lcc3d",
                    "-Wl,-rpath," + libdir], check=True)

    def run(lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True,
                             check=True).stdout
        return [[int(v) for v in line.split()] for line in out.splitlines()]
    return run


def attention(n=1, frame=1, t=1, total=1, heads=1, kv=1, d=64, window=0, sinks=0, ring=0, slots=None,
              k_frames=None, q_frames=None):
    """A probe line from a GPU test's case (and its defaults)."""
    most = max(max(k_frames) if k_frames else total, 1)
    slots = slots or (sinks + ring if ring else most)
    return (f"a {n} {heads} {kv} {d} {frame} {t} {slots} {window} {sinks} {ring} {total} "
            f"{1 if k_frames else 0}")


def launches(row):
    """[(kernel, split, tiles of a frame, tiles)] of an output line."""
    assert len(row) == 1 + 4 * row[0]
    return [tuple(row[1 + 4 * i:5 + 4 * i]) for i in range(row[0])]


def linear(m, n, k, fp8, act=cc3d.ACT_GELU_TANH):
    return f"l {m} {n} {k} {act} {int(fp8)}"


def test_gpu_cases_take_the_kernels_they_are_for(probe):
    out = probe([attention(**kw) for _, _, kw in KERNELS.values()])
    for (name, (kernel, split, _)), row in zip(KERNELS.items(), out):
        assert [x[:2] for x in launches(row)] == [(kernel, split)], name
    assert {(k, s > 1) for k, s, _ in KERNELS.values()} == {
        (k, many) for k in range(8) for many in (False, True)}


def test_cases_whose_waits_run_out_are_splits_and_pairs_of_ctas(probe):
    def case(t, total, frame=1, **kw):
        return attention(t=t // frame, total=total // frame, frame=frame, **kw)
    rows = [launches(r) for r in probe([case(**kw) for kw in (SPLITS | PAIRS).values()])]
    got = {name: (len(r), *r[0][:2]) for name, r in zip(SPLITS | PAIRS, rows)}
    assert all(n == 1 for n, _, _ in got.values()), got
    assert all(got[name][2] > 1 for name in SPLITS), got
    assert {got[name][1] for name in SPLITS} >= {1, 4, 5, 6, 7}, got
    assert {got[name][1:] for name in PAIRS} == {(2, 1), (3, 1)}, got


def test_long_frames_go_in_two_launches(probe):
    """(What the GPU test of them leaves open.)"""
    got = {name: row[0] for name, row in
           zip(LONG_FRAMES, probe([attention(**kw) for _, kw in LONG_FRAMES.values()]))}
    assert all(got[name] >= least for name, (least, _) in LONG_FRAMES.items())
    assert got["ring with sink"] == got["many heads"] == 2


def test_gpu_sizes_take_every_tile_and_split_of_the_product(probe):
    for fp8 in (False, True):
        out = probe([linear(*size, fp8) for size in CHOICES])
        assert {(pair, nt) for few, pair, nt, _, _ in out if not few} == {
            (0, 64), (0, 128), (1, 128), (1, 256)}
        few = [row for row in out if row[0]]
        assert {row[2] for row in few} == set(range(16, 129, 16))
        assert {row[4] for row in few} >= {1, 2, 3, 4, 5, 6, 8}


def test_choices_cover_the_call(probe):
    """Query tiles of all launches cover the chunk, no CTA of a cluster is sure
    to have no keys, head sizes fit the kernel."""
    rng = random.Random(5)
    rows_of = [256, 256, 128, 128, 128, 128, 128, 128]
    keys_of = [64, 64, 64, 64, 128, 128, 64, 64]
    most = [64, 128, 64, 128, 64, 128, 256, 384]
    calls = []
    for _ in range(3000):
        frame = rng.choice((1, 1, 7, 64, 130, 1560))
        t = rng.randint(1, 5) if frame > 1 else rng.choice((1, 2, 50, 700, 8190))
        kv, group = rng.choice((1, 2, 5, 16)), rng.choice((1, 2, 3, 8, 40, 128))
        calls.append(dict(n=rng.choice((1, 3, 16)), frame=frame, t=t, total=rng.choice((0, t, t + 900)),
                          heads=kv * group, kv=kv, d=8 * rng.randint(1, 48),
                          window=rng.choice((0, 1, 6, 300)), sinks=rng.choice((0, 1, 9))))
    for kw, row in zip(calls, probe([attention(**kw) for kw in calls])):
        assert 1 <= row[0] <= 2, kw
        done, tok_tile = 0, 128 // (kw["heads"] // kw["kv"])
        for kernel, split, per_frame, tiles in launches(row):
            rows = rows_of[kernel] // 128 * tok_tile
            assert 1 <= split <= 8 and kw["d"] <= most[kernel], kw
            assert done % rows == 0, kw
            if per_frame:
                assert tiles == per_frame * kw["t"] and per_frame * rows >= kw["frame"], kw
                done = kw["t"] * kw["frame"]
            else:
                done += tiles * rows
            assert split == 1 or split <= -(-max(kw["total"], 1) * kw["frame"] // keys_of[kernel]), kw
        assert done >= kw["t"] * kw["frame"], kw


def test_choices_that_the_timed_cases_rest_on(probe):
    token = attention(n=8, total=20000, heads=32, kv=8, d=128, window=8192, sinks=16, ring=8192,
                      k_frames=[20000] * 8)
    prompt = attention(t=8190, total=8190, heads=16, kv=4, d=128, window=2048, sinks=4)
    frames = attention(frame=1560, t=5, total=5, d=384, window=1)
    stream = attention(frame=1560, total=21, heads=12, kv=12, d=128, window=6, sinks=1, ring=6)
    got = [[x[:2] for x in launches(row)] for row in probe([token, prompt, frames, stream])]
    assert got == [[(5, 2)], [(1, 1)], [(7, 2)], [(1, 2), (5, 8)]]
    # the mid-block's q, k, v product; a wide feed-forward's two; one row
    out = probe([linear(7800, 1152, 384, False, 0), linear(8190, 2048, 8192, False, 0),
                 linear(7800, 8192, 2048, True), linear(1, 12288, 2048, False, cc3d.ACT_SILU)])
    assert [row[:3] for row in out] == [[0, 1, 128], [0, 1, 256], [0, 1, 256], [1, 0, 16]]
