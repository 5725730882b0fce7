"""The attention reference itself, the paged index arithmetic the kernels share (compiled for
the host), and the entry points' refusals: all without a GPU."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import attn_ref as R
from gated_deltanet_sequence_delta_b200 import binding, build as gbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ---- the reference -----------------------------------------------------------------
def test_two_keys_by_hand():
    """q = 1, k = (0, ln 3), v = (4, 8): weights 1/4 and 3/4, so 4/4 + 24/4 = 7."""
    o, A, _ = R.attend_row(np.array([1.0]), np.array([[0.0], [np.log(3.0)]]), np.array([[4.0], [8.0]]), 1.0)
    assert abs(o[0] - 7.0) < 1e-12 and abs(A[0] - 7.0) < 1e-12


def test_causal_grouped_and_empty_rows():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(5, 2, 8)), rng.normal(size=(5, 2, 8))
    o, _ = R.attention(q, k, v, 2, 0.3, "fp32")
    # the last row by a dense product; head 3 reads key-value head 1
    s = 0.3 * k[:, 1] @ q[2, 3]
    np.testing.assert_allclose(o[2, 3], np.exp(s) @ v[:, 1] / np.exp(s).sum(), rtol=1e-12)
    # a row's later keys do not matter to it
    v2 = v.copy()
    v2[3:] = 1e9
    np.testing.assert_allclose(R.attention(q, k, v2, 2, 0.3, "fp32")[0][0], o[0], rtol=1e-12)
    # past < 0: leading rows see nothing
    o, b = R.attention(q, k[:1], v[:1], -2, 0.3, "fp32")
    assert not o[:2].any() and not b[:2].any()
    np.testing.assert_allclose(o[2, 0], v[0, 0])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_relative_position(interleaved):
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=16), rng.normal(size=16)
    f = np.array([1.0, 0.3, 0.01])
    d = [R.rotate(q, a, f, interleaved) @ R.rotate(k, b, f, interleaved) for a, b in ((7, 3), (1007, 1003))]
    assert abs(d[0] - d[1]) < 1e-9
    y = R.rotate(q, 5, f, interleaved)
    assert abs(np.linalg.norm(y) - np.linalg.norm(q)) < 1e-12 and (y[6:] == q[6:]).all()


# ---- paged.cuh on the host ------------------------------------------------------------
@pytest.fixture(scope="module")
def paged(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged")
    src = d / "paged_host.cpp"
    src.write_text('''
#include "paged.cuh"
extern "C" void rows(const int32_t* cu, const int32_t* lens, int n, int64_t nq, int64_t nt, int64_t mx, int* out) {
    const gdn::SeqRows r = gdn::seq_rows(cu, lens, n, nq, nt, mx);
    out[0] = r.q0; out[1] = r.n_q; out[2] = r.n_kv; out[3] = r.bad;
}
extern "C" int64_t row(const int32_t* table, int64_t pos, int shift, int n_pages) {
    return gdn::cache_row(table, pos, shift, n_pages);
}
''')
    so = d / "paged_host.so"
    inc = os.path.join(ROOT, "gated_deltanet_sequence_delta_b200", "csrc")
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-std=c++17", "-I", inc, "-o", str(so), str(src)], check=True)
    L = ctypes.CDLL(str(so))
    L.row.restype = ctypes.c_int64
    return L


def _rows(L, cu, lens, n, nq=0, nt=100, mx=1000):
    i32 = ctypes.c_int32
    out = (ctypes.c_int * 4)()
    c = None if cu is None else (i32 * len(cu))(*cu)
    k = None if lens is None else (i32 * len(lens))(*lens)
    L.rows(c, k, n, ctypes.c_int64(nq), ctypes.c_int64(nt), ctypes.c_int64(mx), out)
    return tuple(out)


def test_sequence_rows(paged):
    assert _rows(paged, [0, 3, 10], None, 1) == (3, 7, 7, 0)
    assert _rows(paged, [0, 3, 10], [5, 40], 1) == (3, 7, 40, 0)
    assert _rows(paged, [0, 3, 10], [5, 2], 1) == (3, 7, 2, 0)          # shorter than its new tokens
    assert _rows(paged, None, None, 2, nq=25) == (50, 25, 25, 0)        # dense
    assert _rows(paged, None, [9, 0, 4], 1, nq=1) == (1, 1, 0, 0)       # an idle slot
    # bad tables: skipped, with the finding's code
    assert _rows(paged, [0, 30, 10], None, 1) == (0, 0, 0, 1)           # decreasing
    assert _rows(paged, [0, 3, 101], None, 1) == (0, 0, 0, 1)           # past the last row
    assert _rows(paged, [-4, 3], None, 0) == (0, 0, 0, 1)
    assert _rows(paged, [2, 3], None, 0) == (0, 0, 0, 1)                # does not start at 0
    assert _rows(paged, [0, 3], [-1], 0) == (0, 0, 0, 3)
    assert _rows(paged, [0, 3], [1001], 0) == (0, 0, 0, 3)              # longer than its table row
    assert _rows(paged, [0, 3], [1000], 0) == (0, 3, 1000, 0)
    assert _rows(paged, [0, 2 ** 31 - 1], None, 0) == (0, 0, 0, 1)


def test_cache_rows(paged):
    t = (ctypes.c_int32 * 4)(5, -1, 7, 2 ** 31 - 1)
    row = lambda pos, shift=4, n=8: paged.row(t, ctypes.c_int64(pos), shift, n)
    assert row(0) == 80 and row(15) == 95 and row(33) == 7 * 16 + 1
    assert row(16) == -1 and row(48) == -1                              # no such page
    assert row(33, n=7) == -1                                           # page n_pages
    big = (ctypes.c_int32 * 1)(2 ** 24 - 1)                             # row numbers near 2^31
    assert paged.row(big, ctypes.c_int64(127), 7, 2 ** 24) == 2 ** 31 - 1


# ---- refusals -------------------------------------------------------------------------
A = 0x7f0000000000          # fake, 16-byte aligned device addresses: never dereferenced
MB = 1 << 20


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return binding.lib()


def _append(L, **kw):
    a = dict(q=A, k=A + 16 * MB, v=A + 32 * MB, io=1, qs=1024, ks=256, vs=256, f=A + 48 * MB, rot=64, il=0,
             cu=A + 49 * MB, lens=A + 50 * MB, table=A + 51 * MB, T=100, N=3, HQ=8, HKV=2, D=128, n_pages=64, page=16,
             width=20, qo=A + 64 * MB, kc=A + 128 * MB, vc=A + 192 * MB)
    a.update(kw)
    return L.gdn_attn_append(a["q"], a["k"], a["v"], a["io"], a["qs"], a["ks"], a["vs"], a["f"], a["rot"], a["il"],
                             a["cu"], a["lens"], a["table"], a["T"], a["N"], a["HQ"], a["HKV"], a["D"], a["n_pages"],
                             a["page"], a["width"], a["qo"], a["kc"], a["vc"], None)


def test_append_refusals(L):
    for name in ("k", "v", "lens", "table", "kc", "vc", "f"):
        assert _append(L, **{name: None}) == 1, name
    assert _append(L, q=None) == 1                          # q_out without q
    assert _append(L, qo=None) == 1
    assert _append(L, cu=None) == 2                         # one token per sequence: T == N
    assert _append(L, HQ=7) == 2 and _append(L, HKV=0) == 2 and _append(L, T=-1) == 2 and _append(L, N=-1) == 2
    assert _append(L, rot=144) == 2 and _append(L, rot=-16) == 2
    assert _append(L, rot=24) == 4                          # not a multiple of 16
    assert _append(L, D=96, qs=768, ks=192, vs=192) == 4
    assert _append(L, io=2) == 4
    assert _append(L, page=8) == 4 and _append(L, page=48) == 4 and _append(L, page=256) == 4
    assert _append(L, page=0) == 2
    assert _append(L, n_pages=1 << 27) == 4                 # row numbers past 32 bits
    assert _append(L, qs=1023) == 2 and _append(L, ks=128) == 2
    assert _append(L, qs=1028) == 3                         # token stride not a multiple of 16 bytes
    assert _append(L, k=A + 16 * MB + 8) == 3
    assert _append(L, kc=A) == 5                            # cache over q
    assert _append(L, kc=A + 128 * MB, vc=A + 128 * MB + 4096) == 5
    assert _append(L, qo=A + 2048) == 5                     # q_out over q, not in place
    assert _append(L, qo=A, qs=2048) == 5                   # in place only where q is contiguous
    assert _append(L, qo=A + 16 * MB) == 5                  # q_out over k
    assert _append(L, T=0, cu=A + 49 * MB) == 0             # nothing to do
    assert _append(L, N=0) == 0


def _prefill(L, **kw):
    a = dict(q=A, k=A + 16 * MB, v=A + 32 * MB, io=1, cu=None, B=2, T=100, N=2, HQ=8, HKV=2, D=128, scale=0.1, z=None,
             o=A + 48 * MB, ws=A + 1024 * MB, nws=512 * MB)
    a.update(kw)
    return L.gdn_attn_prefill(a["q"], a["k"], a["v"], a["io"], a["cu"], a["B"], a["T"], a["N"], a["HQ"], a["HKV"],
                              a["D"], a["scale"], a["z"], a["o"], a["ws"], a["nws"], None)


def test_prefill_refusals(L):
    for name in ("q", "k", "v", "o"):
        assert _prefill(L, **{name: None}) == 1, name
    assert _prefill(L, N=1) == 2 and _prefill(L, cu=A + 80 * MB) == 2 and _prefill(L, T=-1) == 2
    assert _prefill(L, HQ=9) == 2 and _prefill(L, T=2 ** 31) == 2 and _prefill(L, T=2 ** 30) == 2
    assert _prefill(L, scale=float("nan")) == 2 and _prefill(L, scale=float("inf")) == 2
    assert _prefill(L, D=256) == 4 and _prefill(L, io=3) == 4 and _prefill(L, HQ=2048) == 4
    assert _prefill(L, ws=None) == 6 and _prefill(L, nws=16) == 6
    assert _prefill(L, z=A + 90 * MB + 2) == 3 and _prefill(L, q=A + 4) == 3
    assert _prefill(L, o=A) == 5 and _prefill(L, z=A + 48 * MB + 16) == 5 and _prefill(L, ws=A + 16 * MB) == 5
    assert _prefill(L, T=0) == 0 and _prefill(L, B=0, N=0) == 0
    assert L.gdn_attn_prefill_workspace_bytes(1000, 3, 8, 2, 128, 1) >= 256
    assert L.gdn_attn_prefill_workspace_bytes(1000, 3, 8, 3, 128, 1) == 0
    assert L.gdn_attn_prefill_workspace_bytes(2 ** 31, 3, 8, 2, 128, 1) == 0


def _paged_call(L, **kw):
    a = dict(q=A, io=1, kc=A + 16 * MB, vc=A + 32 * MB, table=A + 100 * MB, lens=A + 101 * MB, cu=A + 102 * MB, T=100,
             N=2, HQ=8, HKV=2, D=128, n_pages=64, page=16, width=20, scale=0.1, z=None, o=A + 48 * MB, ws=A + 1024 * MB,
             nws=512 * MB)
    a.update(kw)
    return L.gdn_attn_prefill_paged(a["q"], a["io"], a["kc"], a["vc"], a["table"], a["lens"], a["cu"], a["T"], a["N"],
                                    a["HQ"], a["HKV"], a["D"], a["n_pages"], a["page"], a["width"], a["scale"],
                                    a["z"], a["o"], a["ws"], a["nws"], None)


def _decode(L, **kw):
    a = dict(q=A, io=1, kc=A + 16 * MB, vc=A + 32 * MB, table=A + 100 * MB, lens=A + 101 * MB, B=4, HQ=8, HKV=2,
             D=128, n_pages=64, page=16, width=20, scale=0.1, z=None, o=A + 48 * MB, ws=A + 64 * MB, nws=8 * MB)
    a.update(kw)
    return L.gdn_attn_decode(a["q"], a["io"], a["kc"], a["vc"], a["table"], a["lens"], a["B"], a["HQ"], a["HKV"],
                             a["D"], a["n_pages"], a["page"], a["width"], a["scale"], a["z"], a["o"], a["ws"],
                             a["nws"], None)


@pytest.mark.parametrize("call", [_paged_call, _decode])
def test_paged_refusals(L, call):
    for name in ("q", "kc", "vc", "o", "table", "lens"):
        assert call(L, **{name: None}) == 1, name
    assert call(L, HQ=9) == 2 and call(L, page=-16) == 2 and call(L, width=-1) == 2
    assert call(L, scale=float("nan")) == 2
    assert call(L, D=32) == 4 and call(L, page=24) == 4 and call(L, n_pages=2 ** 27) == 4 and call(L, io=7) == 4
    assert call(L, width=2 ** 27) == 4
    assert call(L, ws=None) == 6 and call(L, nws=8) == 6
    assert call(L, table=A + 100 * MB + 4) == 3
    assert call(L, o=A + 16 * MB) == 5 and call(L, ws=A + 101 * MB) == 5 and call(L, o=A + 100 * MB) == 5


@pytest.mark.parametrize("call", [_paged_call, _decode])
def test_a_cache_without_pages_is_refused(L, call):
    assert call(L, n_pages=0) == 2 and call(L, n_pages=-1) == 2


@pytest.mark.parametrize("call", [_paged_call, _decode])
def test_table_rows_near_the_end_of_32_bits(L, call):
    """The kernels' look past a context's last position stays within 32 bits: a table row may hold 2^31 - 256
    positions (the call then gets as far as its workspace), and no more."""
    most = 2 ** 31 - 256
    for page in (16, 128):
        assert call(L, page=page, width=most // page, ws=None) == 6
        assert call(L, page=page, width=most // page + 1) == 4
    assert _append(L, width=most // 16 + 1) == 4


def test_tokens_near_the_end_of_32_bits(L):
    size = lambda n: L.gdn_attn_prefill_workspace_bytes(n, 1, 1, 1, 64, 1)
    assert size(2 ** 31 - 256) > 0 and size(2 ** 31 - 255) == 0
    assert _prefill(L, B=1, N=1, T=2 ** 31 - 255, HQ=1, HKV=1) == 4


def test_sequences_past_what_the_lists_count(L):
    """Rows to do again are listed in records counted in 32 bits, 16 a key-value head and tile."""
    size = lambda n: L.gdn_attn_prefill_workspace_bytes(1, n, 8, 8, 64, 1)
    assert size(2 ** 24 - 2) > 0 and size(2 ** 24 - 1) == 0 and size(2 ** 27) == 0
    assert _paged_call(L, T=1, N=2 ** 24 - 1, HQ=8, HKV=8, D=64) == 4


def test_paged_nothing_to_do_and_status(L):
    assert _paged_call(L, cu=None) == 1
    assert _paged_call(L, T=0) == 0 and _paged_call(L, N=0) == 0 and _decode(L, B=0) == 0 and _decode(L, B=-1) == 2
    assert L.gdn_attn_decode_workspace_bytes(64, 32, 8, 128, 1) >= 256
    assert L.gdn_attn_decode_workspace_bytes(64, 32, 7, 128, 1) == 0
    assert L.gdn_attn_status(None) == 1
