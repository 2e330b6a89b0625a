"""Host-side refusals of the queries' and keys' norms and of the paged caches: argument validation runs before any CUDA
call, so made-up addresses serve as pointers here.  And the fp64 definitions against one another."""
import ctypes

import numpy as np
import pytest
import torch

import linear_attention_recurrence_chunked_gb300 as la
from linear_attention_recurrence_chunked_gb300 import _build
from tests import paged_oracle as ref

BASE = 0x100000
T = la.LATensor
INV, UNS, WS = la.LA_ERR_INVALID_ARGUMENT, la.LA_ERR_UNSUPPORTED, la.LA_ERR_WORKSPACE
BF, FP = la.LA_DTYPE_BF16, la.LA_DTYPE_F32


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return la.load_library()


def at(k):
    return BASE + (k << 20)


def made(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def qk_args(**kw):
    B, H, Hkv, N, d = 2, 4, 2, 10, 64
    x = lambda k, h: T(at(k), h * N * d, N * d, d)  # noqa: E731
    return made(la.QkNormRopeArgs(B, H, Hkv, N, d, 32, 100, BF, BF, FP, 1, x(0, H), x(1, Hkv), x(2, H), x(3, Hkv), at(4), at(5),
                                  at(6), at(7), at(8), at(9), 1e-6, 0, 0, 1), kw)


def append_args(**kw):
    B, H, N, d = 2, 2, 10, 64
    x = lambda k: T(at(k), H * N * d, N * d, d)  # noqa: E731
    return made(la.PagedAppendArgs(B, H, N, d, 32, 100, 16, 30, 5, BF, 0, x(0), x(1), at(2), at(3), at(4), at(5), at(6), at(7),
                                   at(8), 0), kw)


def read_args(**kw):
    B, H, N, d = 2, 2, 10, 64
    x = lambda k: T(at(k), H * N * d, N * d, d)  # noqa: E731
    return made(la.PagedReadArgs(B, H, N, d, 16, 30, 5, BF, BF, 0, 1, x(0), x(1), at(2), at(3), at(4), at(5)), kw)


def step_args(**kw):
    S, H, d = 3, 4, 64
    x = lambda k: T(at(k), H * d, d, 0)  # noqa: E731
    return made(la.PagedDecodeArgs(S, H, 2, d, 0, 16, 30, 5, BF, BF, 0, 0.125, 0.0, x(0), x(1), at(2), at(3), at(4), at(5), at(6)), kw)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INV), (dict(N=1 << 41), INV), (dict(in_dtype=3), INV), (dict(w_dtype=2), INV), (dict(norm=3), INV), (dict(norm=-1), INV),
    (dict(eps=0.0), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(norm=0), INV), (dict(d=60), UNS), (dict(d=264), UNS),
    (dict(d=0), UNS), (dict(rot=8), UNS), (dict(rot=80), INV), (dict(rot=-16), INV), (dict(cos=None), INV), (dict(sin=None), INV),
    (dict(cos=at(6) + 4), INV), (dict(positions=-1), INV), (dict(q=T(None, 2560, 640, 64)), INV), (dict(q=T(at(0) + 2, 2560, 640, 64)), INV),
    (dict(k=T(at(1), 1280, 640, 63)), INV), (dict(q_out=T(at(2), 0, 640, 64)), INV), (dict(k_out=T(at(3), 1280, 0, 64)), INV),
    (dict(q_out=T(at(0), 5120, 1280, 128)), INV), (dict(q_out=T(at(0), 2560, 640, 64), out_dtype=FP), INV), (dict(q_weight=at(4) + 8), INV),
    (dict(pos=at(8) + 4), INV), (dict(lens=at(9) + 4), INV),
    (dict(B=1 << 30, N=1 << 20), UNS), (dict(k=T(at(1), 1 << 35, 640, 64)), UNS), (dict(q_out=T(at(2), 2560, 1 << 35, 64)), UNS),
    (dict(H=1 << 31), UNS), (dict(B=0), la.LA_OK), (dict(N=0), la.LA_OK), (dict(H=0, H_kv=0), la.LA_OK)])
def test_qk_norm_rope_refusals(lib, kw, status):
    assert lib.la_qk_norm_rope(ctypes.byref(qk_args(**kw)), None) == status


PAGES = [
    (dict(H_kv=-1), INV), (dict(pages=-1), INV), (dict(width=-1), INV), (dict(bits=8), INV), (dict(in_dtype=5), INV), (dict(d=60), UNS),
    (dict(d=136), UNS), (dict(d=0), UNS), (dict(bits=4, in_dtype=FP), UNS), (dict(bits=4, d=96), UNS), (dict(page=0), UNS), (dict(page=8), UNS),
    (dict(page=24), UNS), (dict(page=4112), UNS), (dict(pages=1 << 31), UNS), (dict(width=1 << 30), UNS), (dict(k_pages=None), INV),
    (dict(v_pages=at(3) + 8), INV), (dict(table=None), INV), (dict(table=at(4) + 2), INV)]


@pytest.mark.parametrize("kw,status", PAGES + [
    (dict(B=-1), INV), (dict(N=1 << 41), INV), (dict(rot=8), UNS), (dict(rot=-16), INV), (dict(rot=80), INV), (dict(cos=None), INV),
    (dict(seen=None), INV), (dict(seen=at(5) + 4), INV), (dict(lens=at(8) + 4), INV), (dict(k=T(None, 1280, 640, 64)), INV),
    (dict(v=T(at(1), 1280, 640, 32)), INV), (dict(B=1 << 20, N=1 << 12, width=1), UNS), (dict(v=T(at(1), 1 << 35, 640, 64)), UNS),
    (dict(B=0), la.LA_OK), (dict(N=0), la.LA_OK), (dict(H_kv=0), la.LA_OK)])
def test_paged_append_refusals(lib, kw, status):
    assert lib.la_paged_append(ctypes.byref(append_args(**kw)), None) == status


@pytest.mark.parametrize("kw,status", PAGES + [
    (dict(B=-1), INV), (dict(N=-1), INV), (dict(out_dtype=2), INV), (dict(k=T(at(0), 0, 640, 64)), INV), (dict(v=T(at(1) + 4, 1280, 640, 64)), INV),
    (dict(lens=at(5) + 4), INV), (dict(N=1 << 31), UNS), (dict(B=1 << 24, N=1 << 12, width=1), UNS), (dict(B=0), la.LA_OK), (dict(N=0), la.LA_OK)])
def test_paged_read_refusals(lib, kw, status):
    assert lib.la_paged_read(ctypes.byref(read_args(**kw)), None) == status


@pytest.mark.parametrize("kw,status", PAGES + [
    (dict(S=-1), INV), (dict(H_kv=0), INV), (dict(H_kv=3), INV), (dict(H=34), UNS), (dict(window=-1), INV), (dict(out_dtype=2), INV),
    (dict(softcap=-1.0), INV), (dict(softcap=float("nan")), INV), (dict(softcap=1e38), INV), (dict(q=T(None, 256, 64, 0)), INV),
    (dict(q=T(at(0) + 2, 256, 64, 0)), INV), (dict(q=T(at(0), 256, 60, 0)), INV), (dict(out=T(at(1), 0, 64, 0)), INV),
    (dict(out=T(at(1), 256, 0, 0)), INV), (dict(lens=None), INV), (dict(lens=at(5) + 4), INV), (dict(slopes=at(6) + 2), INV),
    (dict(S=1 << 22), UNS), (dict(S=0), la.LA_OK), (dict(H=0), la.LA_OK)])
def test_paged_decode_refusals(lib, kw, status):
    assert lib.la_paged_decode_step(ctypes.byref(step_args(**kw)), None, 0, None) == status


def test_paged_decode_workspace(lib):
    long = dict(width=1000)
    need = lib.la_paged_decode_workspace_size(ctypes.byref(step_args(**long)))
    assert need > 0 and need % (3 * 4 * 66 * 4) == 0
    assert lib.la_paged_decode_workspace_size(ctypes.byref(step_args())) == 0  # 80 tokens are one part
    assert lib.la_paged_decode_workspace_size(ctypes.byref(step_args(window=100, **long))) == 0
    assert lib.la_paged_decode_workspace_size(ctypes.byref(step_args(H_kv=0))) == 0
    assert lib.la_paged_decode_workspace_size(ctypes.byref(step_args(S=0, **long))) == 0
    assert lib.la_paged_decode_workspace_size(None) == 0
    for ws, size in ((None, need), (at(20), need - 1), (at(20) + 8, need)):
        assert lib.la_paged_decode_step(ctypes.byref(step_args(**long)), ws, size, None) == WS


def test_null_arguments(lib):
    for fn in (lib.la_qk_norm_rope, lib.la_paged_append, lib.la_paged_read):
        assert fn(None, None) == INV
    assert lib.la_paged_decode_step(None, None, 0, None) == INV


def test_binding_refuses(lib):
    x, pages, table, one = torch.zeros((1, 2, 4, 64)), torch.zeros((3, 2, 16, 64)), torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    for call in (lambda: la.la_qk_norm_rope(x), lambda: la.la_qk_norm_rope(x, x[0]), lambda: la.la_qk_norm_rope(x, norm="mean"),
                 lambda: la.la_qk_norm_rope(x, cos=torch.zeros((4, 16))), lambda: la.la_qk_norm_rope(x, cos=torch.zeros((4, 40)), sin=torch.zeros((4, 40))),
                 lambda: la.la_qk_norm_rope(x[0, 0]), lambda: la.la_paged_append(x, x, pages, pages, table, one),
                 lambda: la.la_paged_append(x, x[0], pages, pages, table, one),
                 lambda: la.la_paged_append(x, x, torch.zeros((3, 2, 16, 40), dtype=torch.uint8), pages, table, one),
                 lambda: la.la_paged_append(x, x, pages[0], pages, table, one),
                 lambda: la.la_paged_read(pages, pages, table, one, 4), lambda: la.la_paged_read(pages, pages, table, one, 4, k=x),
                 lambda: la.la_paged_decode_step(x, pages, pages, table, one), lambda: la.la_paged_decode_step(x[:, :, 0], pages, pages, table, one),
                 lambda: la.la_paged_decode_workspace_size(x[:, :, 0, :32], pages, pages, table)):
        with pytest.raises(ValueError):
            call()


def test_packed_arguments_are_the_structures_bytes():
    T4 = lambda k: T(at(k), 1 + k, 2 + k, 3 + k)  # noqa: E731
    W4 = lambda k: (at(k), 1 + k, 2 + k, 3 + k)  # noqa: E731
    A = lambda *ks: tuple(at(k) for k in ks)  # noqa: E731
    cases = [
        (la._QK_NORM_ROPE, la.QkNormRopeArgs(1, 2, 3, 4, 5, 6, 7, 1, 0, 1, 2, *(T4(k) for k in range(4)), *A(4, 5, 6, 7, 8, 9), 0.5, 1, 0, 1),
         (1, 2, 3, 4, 5, 6, 7, 1, 0, 1, 2, *(w for k in range(4) for w in W4(k)), *A(4, 5, 6, 7, 8, 9), 0.5, 1, 0, 1)),
        (la._PAGED_APPEND, la.PagedAppendArgs(1, 2, 3, 4, 5, 6, 7, 8, 9, 1, 4, T4(0), T4(1), *A(2, 3, 4, 5, 6, 7, 8), 1),
         (1, 2, 3, 4, 5, 6, 7, 8, 9, 1, 4, *W4(0), *W4(1), *A(2, 3, 4, 5, 6, 7, 8), 1)),
        (la._PAGED_READ, la.PagedReadArgs(1, 2, 3, 4, 5, 6, 7, 1, 0, 4, 1, T4(0), T4(1), *A(2, 3, 4, 5)),
         (1, 2, 3, 4, 5, 6, 7, 1, 0, 4, 1, *W4(0), *W4(1), *A(2, 3, 4, 5))),
        (la._PAGED_DECODE, la.PagedDecodeArgs(1, 2, 3, 4, 5, 6, 7, 8, 1, 0, 4, 0.5, 2.5, T4(0), T4(1), *A(2, 3, 4, 5, 6)),
         (1, 2, 3, 4, 5, 6, 7, 8, 1, 0, 4, 0.5, 2.5, *W4(0), *W4(1), *A(2, 3, 4, 5, 6))),
    ]
    for packer, struct, words in cases:
        assert packer.size == ctypes.sizeof(struct)
        assert packer.pack(*words) == bytes(struct)


def test_the_rotation_of_the_oracle_keeps_lengths_and_depends_on_distances_alone():
    g = np.random.default_rng(3)
    cos, sin = (t.double().numpy() for t in ref.tables(50, 32))
    for interleaved in (False, True):
        q, k = g.standard_normal(40), g.standard_normal(40)
        at3 = [ref.turn(x, cos[p], sin[p], interleaved)[0] for x, p in ((q, 3), (k, 11))]
        at20 = [ref.turn(x, cos[p], sin[p], interleaved)[0] for x, p in ((q, 20), (k, 28))]
        assert abs(at3[0] @ at3[0] - q @ q) < 1e-5  # the tables are fp32
        assert abs(at3[0] @ at3[1] - at20[0] @ at20[1]) < 1e-5


def test_quantised_rows_of_the_oracle_stand_for_what_they_came_from():
    x = torch.randn((3, 128), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).double().numpy()
    q, scale, lo = ref.quantise(x)
    back = np.repeat(lo, 64, -1) + np.repeat(scale, 64, -1) * np.clip(np.rint(q), 0, 15)
    # half a step, and at the largest the bf16 scale's rounding times 15 codes
    assert np.all(np.abs(back - x) <= np.repeat(scale, 64, -1) * (0.5 + 15 * 2.0 ** -8))
