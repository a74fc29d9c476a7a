"""The paged KV cache without a GPU: the index arithmetic of the kernels (csrc/paged_map.h, compiled here
for the CPU) stays inside its buffers whatever lengths, pages and starts the device holds; the 4-bit row
format; and the refusals of the entry points, which come before any CUDA call."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import long_context_sparse_spa_b200 as spa
from long_context_sparse_spa_b200 import _abi
from oracle import paged as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SHIM = r"""
#include "paged_map.h"
using namespace spa;
extern "C" {
static PagedView view(int np, int H, int sh, int d, int B, int mp, int i4) {
    PagedView v{}; v.num_pages = np; v.Hkv = H; v.page_shift = sh; v.d = d; v.B = B; v.max_pages = mp; v.int4 = i4;
    v.row_bytes = paged_row_bytes(i4, d); return v;
}
long long t_slot(int B, int mp, int sh, int b, long long n) { return paged_slot(view(1, 1, sh, 64, B, mp, 1), b, n); }
long long t_row(int np, int H, int sh, int d, int i4, int pid, int g, long long n) {
    return paged_row(view(np, H, sh, d, 1, 1, i4), pid, g, n);
}
int t_len(int mp, int sh, int len, int* bad) {
    bool b = false; int r = paged_len(view(1, 1, sh, 64, 1, mp, 1), len, &b); *bad = b; return r;
}
int t_seq(const int* s, int B, int t) { return paged_seq_of(s, B, t); }
int t_key(int d, int c) { return int4_key_nibble(d, c); }
int t_val(int d, int c) { return int4_value_nibble(d, c); }
int t_lim(int len, int n, int TQ, int j) { return paged_tile_limit(len, n, TQ, j); }
int t_tq(int rows, int G) { return paged_tokens_per_tile(rows, G); }
int t_owner(long long x, long long TT, int G) { return paged_tile_owner(x, TT, G); }
int t_bytes(int i4, int d) { return paged_row_bytes(i4, d); }
}
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged_map")
    (d / "shim.cpp").write_text(SHIM)
    so = str(d / "shim.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "long_context_sparse_spa_b200", "csrc"), "-o", so, str(d / "shim.cpp")],
                   check=True)
    L = ctypes.CDLL(so)
    i, ll, p = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p
    L.t_slot.restype, L.t_slot.argtypes = ll, [i, i, i, i, ll]
    L.t_row.restype, L.t_row.argtypes = ll, [i, i, i, i, i, i, i, ll]
    L.t_seq.argtypes = [p, i, i]
    L.t_owner.argtypes = [ll, ll, i]
    return L


EXTREMES = [-2**31, -1, 0, 1, 15, 16, 17, 2**31 - 1]


def test_page_and_row_indexes_stay_inside(shim):
    rng = np.random.default_rng(0)
    for _ in range(4000):
        B, mp, sh = int(rng.integers(1, 9)), int(rng.integers(0, 50)), int(rng.integers(4, 11))
        b = int(rng.choice([-1, 0, B - 1, B, int(rng.integers(0, B))]))
        n = int(rng.choice([*EXTREMES, int(rng.integers(0, 60000)), 2**40, -2**40]))
        s = shim.t_slot(B, mp, sh, b, n)
        assert -1 <= s < B * mp
        assert (s >= 0) == (0 <= b < B and 0 <= n < mp << sh)
        np_, H, d, i4 = int(rng.integers(0, 7)), int(rng.integers(1, 9)), int(rng.choice([64, 128])), int(rng.integers(0, 2))
        pid, g = int(rng.choice([*EXTREMES, int(rng.integers(0, 7))])), int(rng.integers(0, H))
        row, size = shim.t_row(np_, H, sh, d, i4, pid, g, max(n, 0)), shim.t_bytes(i4, d)
        assert row == -1 or (0 <= row and row + size <= np_ * H * (size << sh) and row % 16 == 0)
        assert (row >= 0) == (0 <= pid < np_)


def test_row_offsets_pass_32_bits(shim):
    # 40 000 pages of 128 tokens x 8 kv heads x 144 bytes: the last row lies past 2^32 bytes
    assert shim.t_row(40000, 8, 7, 128, 1, 39999, 7, 127) == (40000 * 8 * 128 - 1) * 144 > 2**32


def test_lengths_are_clamped_and_reported(shim):
    bad = ctypes.c_int()
    for mp, sh, ln in [(0, 4, 0), (3, 4, 48), (3, 4, 49), (3, 4, -1), (7, 6, 2**31 - 1), (7, 6, -2**31)]:
        r = shim.t_len(mp, sh, ln, ctypes.byref(bad))
        cap = mp << sh
        assert r == min(max(ln, 0), cap) and bool(bad.value) == (ln < 0 or ln > cap)


def test_sequence_of_a_row(shim):
    start = np.array([2, 2, 5, 5, 9], np.int32)
    got = [shim.t_seq(start.ctypes.data, 4, t) for t in range(11)]
    assert got == [-1, -1, 1, 1, 1, 3, 3, 3, 3, -1, -1]
    assert [shim.t_seq(None, 3, t) for t in range(4)] == [0, 1, 2, -1]
    rng = np.random.default_rng(1)
    for _ in range(2000):   # starts in no order: an answer is still a sequence whose rows hold the token
        s = rng.integers(-2**31, 2**31, int(rng.integers(2, 9))).astype(np.int32)
        t = int(rng.integers(0, 100))
        b = shim.t_seq(s.ctypes.data, len(s) - 1, t)
        assert b == -1 or s[b] <= t < s[b + 1]


@pytest.mark.parametrize("d", [64, 128])
def test_nibble_places_are_a_permutation_and_match_the_format(shim, d):
    kp, vp = ref.nibble_places(d)
    assert [shim.t_key(d, c) for c in range(d)] == kp.tolist() and sorted(kp) == list(range(d))
    assert [shim.t_val(d, c) for c in range(d)] == vp.tolist() and sorted(vp) == list(range(d))


def test_query_tiles_cover_every_query_once(shim):
    for G in (1, 3, 8, 16):
        TQ = shim.t_tq(16, G)
        assert 1 <= TQ and TQ * G <= 16
        for n, ln in [(1, 1), (5, 5), (7, 100), (9, 4), (3, 0)]:
            lims = [shim.t_lim(ln, n, TQ, j) for j in range(-(-n // TQ))]
            assert lims[-1] == ln and lims == [max(0, ln - n + min((j + 1) * TQ, n)) for j in range(len(lims))]


def test_tile_owners_partition_the_tiles(shim):
    for TT, G in [(1, 1), (7, 3), (148, 148), (1000, 148), (10**10, 148)]:
        for c in {0, G // 2, G - 1}:
            lo, hi = TT * c // G, TT * (c + 1) // G
            for x in {lo, hi - 1}:
                assert shim.t_owner(x, TT, G) == c


@pytest.mark.parametrize("d", [64, 128])
def test_quantised_rows_read_back_within_half_a_step(d):
    rng = np.random.default_rng(d)
    x = (rng.standard_normal((200, 2, d)) * np.exp(rng.normal(0, 6, (200, 2, 1)))).astype(np.float32)
    x[0, 0] = 0
    x[1, 0, 3] = np.nan
    x[2, 1, d - 1] = np.inf
    K, V, ks, vs = ref.unpack(ref.pack(x[:, 0], x[:, 1]))
    for y, s, z in ((K, ks, x[:, 0]), (V, vs, x[:, 1])):
        s = np.repeat(s, d // 4, -1)
        fin = ~np.isnan(s)
        assert np.all(np.abs(y - z)[fin] <= s[fin] / 2 * (1 + 2**-20))
        assert np.all(np.isnan(y) == np.isnan(s))
    assert np.isnan(K[1, :d // 4]).all() and not np.isnan(K[1, d // 4:]).any()
    assert np.isnan(V[2, -(d // 4):]).all() and (K[0] == 0).all()


# ------------------------------------------------------------------------------------------- refusals
def _kv(**kw):
    kv = _abi.SpaPagedKv()
    base = dict(format=_abi.SPA_KV_INT4, num_pages=4, Hkv=2, page=16, d=128, B=2, max_pages=2, data=256,
                page_table=256, kv_len=256)
    for k, v in {**base, **kw}.items():
        setattr(kv, k, v)
    return kv


BAD_KV = [(dict(format=2), "INVALID_ARG"), (dict(Hkv=0), "INVALID_ARG"), (dict(B=-1), "INVALID_ARG"),
          (dict(page=24), "UNSUPPORTED_SHAPE"), (dict(page=8), "UNSUPPORTED_SHAPE"), (dict(page=2048), "UNSUPPORTED_SHAPE"),
          (dict(d=96), "UNSUPPORTED_SHAPE"), (dict(data=None), "INVALID_ARG"), (dict(data=264), "UNSUPPORTED_SHAPE"),
          (dict(kv_len=None), "INVALID_ARG"), (dict(page_table=None), "INVALID_ARG"),
          (dict(max_pages=2**28), "UNSUPPORTED_SHAPE"), (dict(B=70000), "UNSUPPORTED_SHAPE")]


def _call(name, args, ws=4096, n=1 << 40):
    return _abi.lib().spa_status_string(getattr(_abi.lib(), name)(ctypes.byref(args), ws, n, None)).decode()


@pytest.mark.parametrize("kw,want", BAD_KV)
def test_a_bad_cache_is_refused_by_every_entry_point(kw, want):
    a = _abi.SpaPagedAppendArgs(kv=_kv(**kw), T=2)
    a.k = a.v = 256
    g = _abi.SpaPagedGatherArgs(kv=_kv(**kw), N=4, K=256, V=256)
    t = _abi.SpaPagedAttendArgs(kv=_kv(**kw), T=2, Hq=4, q=256, out=256)
    for name, x in (("spa_paged_append", a), ("spa_paged_gather", g), ("spa_paged_attend", t)):
        assert _call(name, x) == "SPA_ERR_" + want, name


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), "INVALID_ARG"), (dict(T=3), "INVALID_ARG"), (dict(k=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"),
    (dict(k=258), "UNSUPPORTED_SHAPE"), (dict(k_token_stride=4), "UNSUPPORTED_SHAPE"),
    (dict(v_head_stride=-8), "INVALID_ARG"), (dict(q=256, Hq=0), "INVALID_ARG"), (dict(q=256, Hq=4), "INVALID_ARG"),
    (dict(q=256, Hq=4, q_out=256), "INVALID_ARG"), (dict(q=256, Hq=4, q_out=520), "UNSUPPORTED_SHAPE"),
    (dict(rot=64), "INVALID_ARG"), (dict(rot=-16), "INVALID_ARG"), (dict(rot=144, inv_freq=256), "INVALID_ARG"),
    (dict(rot=24, inv_freq=256), "UNSUPPORTED_SHAPE")])
def test_append_refusals(kw, want):
    a = _abi.SpaPagedAppendArgs(kv=_kv(), **{**dict(T=2, k=256, v=256), **kw})
    assert _call("spa_paged_append", a) == "SPA_ERR_" + want


def test_small_workspaces_are_refused():
    a = _abi.SpaPagedAppendArgs(kv=_kv(), T=2, k=256, v=256)
    assert _call("spa_paged_append", a, n=255) == "SPA_ERR_WORKSPACE_TOO_SMALL"
    g = _abi.SpaPagedGatherArgs(kv=_kv(), N=4, K=256, V=256)
    assert _call("spa_paged_gather", g, n=255) == "SPA_ERR_WORKSPACE_TOO_SMALL"
    t = _abi.SpaPagedAttendArgs(kv=_kv(), T=2, Hq=4, q=256, out=256)
    need = _abi.lib().spa_paged_attend_workspace_bytes(ctypes.byref(t))
    assert need > 256 and _call("spa_paged_attend", t, n=need - 1) == "SPA_ERR_WORKSPACE_TOO_SMALL"
    assert _call("spa_paged_attend", t, ws=None) == "SPA_ERR_INVALID_ARG"


@pytest.mark.parametrize("kw,want", [
    (dict(Hq=5), "INVALID_ARG"), (dict(Hq=0), "INVALID_ARG"), (dict(Hq=34), "UNSUPPORTED_SHAPE"), (dict(T=3), "INVALID_ARG"),
    (dict(q=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(q=264), "UNSUPPORTED_SHAPE"),
    (dict(out=264), "UNSUPPORTED_SHAPE"), (dict(out_f32=264), "UNSUPPORTED_SHAPE"),
    (dict(idx=256), "INVALID_ARG"), (dict(idx=256, count=256, unit_tokens=0), "INVALID_ARG"),
    (dict(idx=256, count=256, unit_tokens=1, cap=-1), "INVALID_ARG"),
    (dict(idx=256, count=256, unit_tokens=1, collapse=2), "INVALID_ARG"),
    (dict(idx=256, count=256, unit_tokens=1, seq_start=256, T=3), "INVALID_ARG")])
def test_attend_refusals(kw, want):
    t = _abi.SpaPagedAttendArgs(kv=_kv(), **{**dict(T=2, Hq=4, q=256, out=256), **kw})
    assert _call("spa_paged_attend", t) == "SPA_ERR_" + want


def test_nothing_to_do_is_no_error():
    assert _call("spa_paged_append", _abi.SpaPagedAppendArgs(kv=_kv(), T=0, seq_start=256)) == "SPA_OK"
    assert _call("spa_paged_append", _abi.SpaPagedAppendArgs(kv=_kv(B=0), T=0)) == "SPA_OK"
    assert _call("spa_paged_gather", _abi.SpaPagedGatherArgs(kv=_kv(), N=0)) == "SPA_OK"
    assert _call("spa_paged_attend", _abi.SpaPagedAttendArgs(kv=_kv(), T=0, Hq=4, seq_start=256)) == "SPA_OK"
    assert _abi.lib().spa_paged_row_bytes(0, 128) == 512 and _abi.lib().spa_paged_row_bytes(1, 64) == 80
    assert _abi.lib().spa_paged_row_bytes(7, 64) == 0


def test_python_refuses_cpu_tensors_and_wrong_types():
    c = torch.zeros(4, 2, 16, 144, dtype=torch.uint8)
    t, n = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        spa.paged_gather(cache=c, page_table=t, kv_len=n, N=4)
    with pytest.raises(TypeError):
        spa.paged_gather(cache=c.float(), page_table=t, kv_len=n, N=4)
    with pytest.raises(ValueError):
        spa.paged_cache(4, 2, 16, 128, fmt=9)


def test_the_paged_kernels_have_their_bits_of_the_stall_hook():
    L = _abi.lib()
    bits = _abi.SPA_TEST_STALL_PAGED_COPY | _abi.SPA_TEST_STALL_PAGED_CHUNK
    assert L.spa_test_stall(bits) == _abi.SPA_OK and L.spa_test_stall(bits | 32) == _abi.SPA_ERR_INVALID_ARG
    assert L.spa_test_stall(0) == _abi.SPA_OK


def test_every_header_of_the_sources_makes_the_library_stale():
    import re

    from long_context_sparse_spa_b200 import build

    deps = {os.path.realpath(f) for f in build._deps()}
    for src in sorted(deps):
        with open(src) as f:
            for name in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
                at = [os.path.join(d, name) for d in (os.path.dirname(src), build.CSRC, build.INCLUDE)]
                found = [os.path.realpath(p) for p in at if os.path.exists(p)]
                assert found and found[0] in deps, f"{os.path.basename(src)} includes {name}"


def test_heads_that_do_not_divide():
    L = _abi.lib()
    for hq in (0, -2, 1, 3):                # kv heads: 2
        t = _abi.SpaPagedAttendArgs(kv=_kv(), T=5, Hq=hq, q=256, out=256, seq_start=256, sm_scale=1.0)
        assert L.spa_paged_attend_workspace_bytes(ctypes.byref(t)) == 0
        assert _call("spa_paged_attend", t) == "SPA_ERR_INVALID_ARG"


def test_heads_that_are_too_many():
    for hq, hkv in ((65536, 4096), (65536, 32768), (1 << 20, 65536)):
        t = _abi.SpaPagedAttendArgs(kv=_kv(Hkv=hkv), T=2, Hq=hq, q=256, out=256)
        assert _call("spa_paged_attend", t) == "SPA_ERR_UNSUPPORTED_SHAPE"


def test_outputs_over_inputs_are_refused():
    # T = 2 tokens of (4 + 2 + 2) heads of 128 in one projection: 4096 bytes of it, q at 1 << 20, k and v behind it
    at = 1 << 20
    for q_out in (at + 16, at + 4096 - 16, at - 16, at + 1024, at + 1536, at + 2048 + 1536):
        a = _abi.SpaPagedAppendArgs(kv=_kv(), T=2, Hq=4, q=at, k=at + 1024, v=at + 1536, q_out=q_out, q_token_stride=1024,
                                    k_token_stride=1024, v_token_stride=1024, q_head_stride=128, k_head_stride=128,
                                    v_head_stride=128)
        assert _call("spa_paged_append", a) == "SPA_ERR_INVALID_ARG", q_out - at
    for kw in (dict(out=at + 1024), dict(out=at - 2032), dict(out_f32=at - 4080), dict(out=at + 2048 + 1008)):
        t = _abi.SpaPagedAttendArgs(kv=_kv(), **{**dict(T=2, Hq=4, q=at, out=1 << 24, q_token_stride=1024, q_head_stride=128), **kw})
        assert _call("spa_paged_attend", t) == "SPA_ERR_INVALID_ARG", kw
