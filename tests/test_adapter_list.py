"""The adapters' token lists on the host: the arithmetic that the kernels share with
this test (``csrc/ss1_adapter_list.h``, compiled here for the CPU) in a model of
their loops, on index arrays in order and out of order, up to the largest M.

Whatever the arrays hold, every entry of the work list and every slot lies inside
its array and every listed token inside [0, M); in ordered arrays each adapter's
tokens are listed once, in order.
"""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sketched_parameter_sharing_amd", "csrc")
THREADS = 256

MODEL = r"""
#include <algorithm>
#include <cstdint>
#include <vector>
#include "ss1_adapter_list.h"
using namespace ss1;
static int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// plan_outer(): table[most][4] and multi[E + 1][4], -7 where nothing was written.
// Returns how many writes fell outside.
extern "C" int plan(const int* seg, const int* ids, int S, int E, int M, int P, int most, int slots, int* table,
                    int* multi) {
    int outside = 0;
    const auto put = [&](int* to, int64_t at, int64_t count, int a, int b, int c, int d) {
        if (at < 0 || at >= count) { ++outside; return; }
        const int v[4] = {a, b, c, d};
        for (int i = 0; i < 4; ++i) to[4 * at + i] = v[i];
    };
    PlanSums done{0, 0, 0};
    for (int e0 = 0; e0 < E; e0 += 256) {
        std::vector<uint32_t> held(256, 0);  // an LDS counter wraps
        for (int s = 0; s < S; ++s) {
            const int64_t e = int64_t(ids[s]) - e0;
            const int b = clampi(seg[s], 0, M), n = clampi(seg[s + 1], b, M) - b;
            if (e >= 0 && e < 256 && e0 + e < E && n > 0) held[e] += n;
        }
        int x = 0, y = 0, z = 0;
        for (int t = 0; t < 256; ++t) {
            const int e = e0 + t, tokens = clampi(static_cast<int>(held[t]), 0, M);
            const int parts = e < E ? parts_of(tokens, P) : 0;
            const int q = done.entries + x, slot = done.slots + y, c = done.several + z;
            const bool several = parts > 1 && slot + parts <= slots;
            for (int i = 0; i < parts; ++i)
                if (q + i < most) {
                    if (several) put(table, q + i, most, e, i * P, part_end(tokens, P, i), slot + i);
                    else put(table, q + i, most, i == 0 ? e : -1, 0, tokens, -1);
                }
            if (parts > 1) put(multi, 1 + c, E + 1, e, several ? parts : 0, several ? slot : 0, 0);
            x += parts; y += parts > 1 ? parts : 0; z += parts > 1;
        }
        done = plan_add(done, {x, y, z}, most, slots);
    }
    for (int q = done.entries; q < most; ++q) put(table, q, most, -1, 0, 0, -1);
    put(multi, 0, E + 1, done.several, 0, 0, 0);
    return outside;
}

// outer_kernel()'s lists of one part: runs of tokens [first, last) in order.
// Returns their number, -1 where one falls outside [0, M) or the block's ends do
// not ascend.
extern "C" int runs(const int* seg, const int* ids, int S, int M, int e, int part_from, int part_to, int* out,
                    int room) {
    int listed = 0, found = 0;
    for (int s0 = 0; s0 < S; s0 += 256) {
        int ends[256], starts[256], total = 0;
        for (int t = 0; t < 256; ++t) {
            const int s = s0 + t;
            int b = 0, n = 0;
            if (s < S) {
                b = clampi(seg[s], 0, M);
                n = ids[s] == e ? clampi(seg[s + 1], b, M) - b : 0;
            }
            const ListRun r = list_run(b, n, total, M);
            total = add_capped(total, n, M);
            ends[t] = r.end;
            starts[t] = r.start;
            if (r.end != total || (t > 0 && ends[t] < ends[t - 1])) return -1;
        }
        const int from = std::max(0, part_from - listed), to = std::min(total, part_to - listed);
        listed = add_capped(listed, total, M);
        for (int t = 0; t < 256; ++t) {
            const int lo = std::max(from, t > 0 ? ends[t - 1] : 0), hi = std::min(to, ends[t]);
            if (lo >= hi) continue;
            const int64_t a = int64_t(starts[t]) + lo, z = int64_t(starts[t]) + hi;
            if (a < 0 || z > M) return -1;
            if (found < room) { out[2 * found] = static_cast<int>(a); out[2 * found + 1] = static_cast<int>(z); }
            ++found;
        }
    }
    return found;
}
"""


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("list")
    (d / "model.cpp").write_text(MODEL)
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-Wall", "-shared", "-fPIC", f"-I{CSRC}", str(d / "model.cpp"),
                    "-o", str(d / "model.so")], check=True)
    lib = ctypes.CDLL(str(d / "model.so"))
    p, i = ctypes.c_void_p, ctypes.c_int
    lib.plan.argtypes = [p, p, i, i, i, i, i, i, p, p]
    lib.runs.argtypes = [p, p, i, i, i, i, i, p, i]
    return lib


def split(M, parts):
    """Part length, as many entries as E adapters may need less E, and slots: outer_split's."""
    P = max(256, (M // parts + 31) // 32 * 32)
    return P, M // P, 2 * M // P


def planned(model, seg, ids, E, M, parts=100):
    seg, ids = np.asarray(seg, np.int64).astype(np.int32), np.asarray(ids, np.int32)
    P, more, slots = split(M, parts)
    assert M > P and len(seg) == len(ids) + 1
    table, multi = np.full((E + more, 4), -7, np.int32), np.full((E + 1, 4), -7, np.int32)
    outside = model.plan(seg.ctypes.data, ids.ctypes.data, len(ids), E, M, P, E + more, slots, table.ctypes.data,
                         multi.ctypes.data)
    assert outside == 0
    assert (table[:, 0] != -7).all()                                 # every entry is written
    assert ((table[:, 0] >= -1) & (table[:, 0] < E)).all()
    assert ((table[:, 1] >= 0) & (table[:, 1] <= table[:, 2]) & (table[:, 2] <= M)).all()
    assert ((table[:, 3] >= -1) & (table[:, 3] < slots)).all()
    used = table[table[:, 3] >= 0, 3]
    assert len(set(used.tolist())) == len(used)
    several = multi[1:1 + multi[0, 0]]
    assert 0 <= multi[0, 0] <= E and ((several[:, 0] >= 0) & (several[:, 0] < E)).all()
    assert ((several[:, 2] >= 0) & (several[:, 1] >= 0) & (several[:, 2] + several[:, 1] <= slots)).all()
    lists = []
    for e, a, z, _ in table[table[:, 0] >= 0]:
        out = np.zeros((len(ids) + 1, 2), np.int32)
        n = model.runs(seg.ctypes.data, ids.ctypes.data, len(ids), M, int(e), int(a), int(z), out.ctypes.data, len(out))
        assert n >= 0, "a token outside"
        lists.append((int(e), out[:n]))
    return table, multi, lists


def in_order(seg, ids, E, lists):
    """Each adapter's parts, joined, are its segments."""
    for e in range(E):
        got = [(a, z) for k, runs in lists if k == e for a, z in runs.tolist()]
        want = [(a, z) for a, z, i in zip(seg, seg[1:], ids) if i == e and z > a]
        joined = []
        for a, z in got:
            if joined and joined[-1][1] == a:
                joined[-1][1] = z
            else:
                joined.append([a, z])
        merged = []
        for a, z in want:
            if merged and merged[-1][1] == a:
                merged[-1][1] = z
            else:
                merged.append([a, z])
        assert joined == merged, e


TOP = 2 ** 31 - 1


@pytest.mark.parametrize("M,S,E,parts", [(257, 1, 1, 512), (5000, 12, 3, 8), (8192, 24, 6, 20), (100000, 700, 300, 512),
                                         (3 << 20, 1000, 5, 512), (TOP, 40, 2, 512), (TOP, 600, 3, 1), (TOP, 3, 1, 300)])
def test_ordered_offsets_list_every_token_once(model, M, S, E, parts):
    g = np.random.default_rng(M % 1000 + S)
    seg = [0, *sorted(g.integers(0, M, S - 1).tolist()), M]
    ids = g.integers(-1, E, S).tolist()
    if split(M, parts)[0] >= M:  # a single part is the call without a list
        parts = 2
    _, _, lists = planned(model, seg, ids, E, M, parts)
    in_order(seg, ids, E, lists)


@pytest.mark.parametrize("M", [300, 5000, 1 << 23, (1 << 23) + 1, 1 << 24, 1 << 30, TOP])
@pytest.mark.parametrize("kind", ["repeated", "descending", "far outside", "random", "alternating"])
def test_offsets_out_of_order_stay_inside(model, M, kind):
    g = np.random.default_rng(3)
    for S, E in ((1, 1), (256, 1), (257, 3), (700, 300), (2000, 2)):
        seg = {"repeated": np.resize([0, M], S + 1),            # every second segment is all of the batch
               "descending": np.linspace(M, 0, S + 1).astype(np.int64),
               "far outside": g.integers(-2 ** 31, TOP, S + 1),
               "random": g.integers(0, M + 1, S + 1),
               "alternating": np.resize([0, M, M - 1, M], S + 1)}[kind]
        for ids in (np.zeros(S, int), np.arange(S) % E, g.integers(-5, E + 5, S)):
            planned(model, seg, ids, E, M, parts=1 + int(g.integers(2, 512)))


def test_sums_that_pass_their_arrays(model):
    # every adapter with a segment that is the whole batch: many times the entries and slots that there are
    M, E = 1 << 20, 600
    seg = np.resize([0, M], 2 * E + 1)
    planned(model, seg, np.repeat(np.arange(E), 2), E, M, 512)
