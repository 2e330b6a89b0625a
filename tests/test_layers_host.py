"""Host-side refusals of the convolution, scan and attention entry points: argument validation runs before any
CUDA call, so made-up addresses serve as pointers here."""
import ctypes

import pytest
import torch

import linear_attention_recurrence_chunked_gb300 as la
from linear_attention_recurrence_chunked_gb300 import _build

BASE = 0x100000
T = la.LATensor


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return la.load_library()


def at(k):
    return BASE + (k << 20)


def conv_args(**kw):
    B, N, C, W = 2, 10, 64, 4
    a = la.ConvPrefillArgs(B, N, C, W, la.LA_DTYPE_BF16, la.LA_DTYPE_BF16, la.LA_DTYPE_BF16, T(at(0), N * C, 0, C),
                           T(at(1), N * C, 0, C), at(2), at(3), at(4), at(5), None, 1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def conv_step_args(**kw):
    a = la.ConvDecodeArgs(4, 64, 4, la.LA_DTYPE_BF16, la.LA_DTYPE_BF16, la.LA_DTYPE_F32, at(0), 64, at(1), 64, at(2), at(3),
                          at(4), at(4), 1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def ssm_args(**kw):
    B, N, C, n, G = 2, 10, 64, 16, 2
    r = lambda k: T(at(k), N * C, 0, C)  # noqa: E731
    s = lambda k: T(at(k), G * N * n, N * n, n)  # noqa: E731
    a = la.SsmPrefillArgs(B, N, C, n, G, la.LA_DTYPE_BF16, la.LA_DTYPE_BF16, r(0), r(1), r(2), r(3), s(4), s(5), at(6), at(7), at(8),
                          at(9), at(10), None, 1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def ssm_step_args(**kw):
    S, C, n, G = 4, 64, 16, 2
    r = lambda k: T(at(k), C, 0, 0)  # noqa: E731
    s = lambda k: T(at(k), G * n, n, 0)  # noqa: E731
    a = la.SsmDecodeArgs(S, C, n, G, la.LA_DTYPE_BF16, la.LA_DTYPE_BF16, r(0), r(1), r(2), r(3), s(4), s(5), at(6), at(7), at(8), at(9),
                         at(9), 1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def swa_args(**kw):
    B, H, Hkv, N, d = 2, 4, 2, 20, 64
    q = lambda k, h: T(at(k), h * N * d, N * d, d)  # noqa: E731
    a = la.SwaPrefillArgs(B, H, Hkv, N, N, d, 8, la.LA_DTYPE_BF16, la.LA_DTYPE_BF16, q(0, H), q(1, Hkv), q(2, Hkv), q(3, H), 0.125, 0.0,
                          at(4), at(5), at(6), 0, at(7), at(8), at(9))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def swa_step_args(base=None, **kw):
    b = la.SwaDecodeArgs(4, 4, 64, 8, la.LA_DTYPE_BF16, la.LA_DTYPE_BF16, at(0), at(1), at(2), at(3), at(4), at(5), at(6), 0.125)
    for k, v in (base or {}).items():
        setattr(b, k, v)
    a = la.SwaBiasedDecodeArgs(b, 2, 0.0, at(7))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


INV, UNS, WS = la.LA_ERR_INVALID_ARGUMENT, la.LA_ERR_UNSUPPORTED, la.LA_ERR_WORKSPACE
BIG = 1 << 41


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INV), (dict(N=BIG), INV), (dict(in_dtype=7), INV), (dict(w_dtype=2), INV), (dict(W=1), UNS), (dict(W=5), UNS),
    (dict(x=T(None, 640, 0, 64)), INV), (dict(x=T(at(0) + 2, 640, 0, 64)), INV), (dict(x=T(at(0), 640, 0, 60)), INV),
    (dict(x=T(at(0), 640, 0, 0)), INV), (dict(x=T(at(0), -640, 0, 64)), INV), (dict(y=T(at(0), 640, 0, 64)), INV),
    (dict(y=T(at(1), 0, 0, 64)), INV), (dict(w=None), INV), (dict(w=at(2) + 8), INV), (dict(bias=at(3) + 4), INV), (dict(state_out=None), INV),
    (dict(state_in=at(4) + 2), INV), (dict(lens=at(6) + 4), INV), (dict(N=1 << 40, x=T(at(0), 1 << 46, 0, 64), y=T(at(1), 1 << 46, 0, 64)), UNS),
    (dict(B=0), la.LA_OK), (dict(C=0), la.LA_OK)])
def test_conv_prefill_refusals(lib, kw, status):
    assert lib.la_conv_prefill(ctypes.byref(conv_args(**kw)), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), INV), (dict(W=8), UNS), (dict(x=None), INV), (dict(x=at(0) + 4), INV), (dict(x_stride=63), INV), (dict(out_stride=32), INV),
    (dict(out=None), INV), (dict(w=None), INV), (dict(state_in=None), INV), (dict(state_out=None), INV), (dict(out_dtype=9), INV),
    (dict(S=0), la.LA_OK)])
def test_conv_step_refusals(lib, kw, status):
    assert lib.la_conv_decode_step(ctypes.byref(conv_step_args(**kw)), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INV), (dict(G=0), INV), (dict(G=3), INV), (dict(n=0), UNS), (dict(n=65), UNS), (dict(B=65536), UNS),
    (dict(u=T(None, 640, 0, 64)), INV), (dict(delta=T(at(1), 640, 0, 63)), INV), (dict(z=T(at(2) + 8, 640, 0, 64)), INV),
    (dict(y=T(at(3), 0, 0, 64)), INV), (dict(Bm=T(None, 320, 160, 16)), INV), (dict(Bm=T(at(4) + 1, 320, 160, 16)), INV),
    (dict(Cm=T(at(5), 320, -160, 16)), INV), (dict(A=None), INV), (dict(A=at(6) + 2), INV), (dict(D=at(7) + 1), INV), (dict(h_out=None), INV),
    (dict(h_in=at(9) + 4), INV), (dict(lens=at(11) + 4), INV), (dict(in_dtype=5), INV), (dict(B=0), la.LA_OK)])
def test_ssm_prefill_refusals(lib, kw, status):
    assert lib.la_ssm_prefill(ctypes.byref(ssm_args(**kw)), None, 0, None) == status


def test_ssm_workspace(lib):
    long = dict(B=1, N=100000, C=64, G=1, u=T(at(0), 6400000, 0, 64), delta=T(at(1), 6400000, 0, 64), z=T(None, 0, 0, 0),
                y=T(at(3), 6400000, 0, 64), Bm=T(at(4), 1600000, 1600000, 16), Cm=T(at(5), 1600000, 1600000, 16))
    need = lib.la_ssm_prefill_workspace_size(ctypes.byref(ssm_args(**long)))
    assert need > 0
    assert lib.la_ssm_prefill_workspace_size(ctypes.byref(ssm_args())) == 0  # a short prompt is one segment
    assert lib.la_ssm_prefill_workspace_size(ctypes.byref(ssm_args(G=0))) == 0
    assert lib.la_ssm_prefill_workspace_size(None) == 0
    for ws, size in ((None, need), (at(20), need - 1), (at(20) + 8, need)):
        assert lib.la_ssm_prefill(ctypes.byref(ssm_args(**long)), ws, size, None) == WS


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), INV), (dict(G=3), INV), (dict(n=65), UNS), (dict(S=1 << 19), UNS), (dict(u=T(at(0) + 1, 64, 0, 0)), INV),
    (dict(out=T(at(3), 32, 0, 0)), INV), (dict(out=T(None, 64, 0, 0)), INV), (dict(Cm=T(None, 32, 16, 0)), INV), (dict(A=None), INV),
    (dict(state_in=None), INV), (dict(state_out=at(9) + 4), INV), (dict(C=0), la.LA_OK)])
def test_ssm_step_refusals(lib, kw, status):
    assert lib.la_ssm_decode_step(ctypes.byref(ssm_step_args(**kw)), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INV), (dict(H_kv=0), INV), (dict(H_kv=3), INV), (dict(Nq=21), INV), (dict(q_pos0=1), INV), (dict(q_pos0=-1), INV),
    (dict(window=-1), INV), (dict(softcap=-1.0), INV), (dict(softcap=float("nan")), INV), (dict(softcap=float("inf")), INV), (dict(d=60), UNS),
    (dict(d=136), UNS), (dict(d=0), UNS), (dict(k_cache=None), INV), (dict(window=0), UNS), (dict(window=257), UNS),
    (dict(q=T(None, 5120, 1280, 64)), INV), (dict(k=T(at(1) + 2, 2560, 1280, 64)), INV), (dict(v=T(at(2), 2560, 1280, 32)), INV),
    (dict(o=T(at(3), 0, 1280, 64)), INV), (dict(o=T(at(3), 5120, 0, 64)), INV), (dict(slopes=at(4) + 1), INV), (dict(key_lo=at(5) + 2), INV),
    (dict(lens=at(7) + 4), INV), (dict(v_cache=at(9) + 8), INV), (dict(Nk=(1 << 31) - 100), UNS), (dict(in_dtype=3), INV), (dict(B=0), la.LA_OK)])
def test_swa_prefill_refusals(lib, kw, status):
    assert lib.la_swa_prefill(ctypes.byref(swa_args(**kw)), None) == status


@pytest.mark.parametrize("base,kw,status", [
    (dict(S=-1), {}, INV), ({}, dict(H_kv=3), INV), ({}, dict(H_kv=0), INV), (dict(H=34), dict(H_kv=2), UNS), (dict(window=257), {}, UNS),
    (dict(window=0), {}, UNS), (dict(d=12), {}, UNS), (dict(q=None), {}, INV), (dict(k_cache=at(3) + 8), {}, INV), (dict(pos=None), {}, INV),
    ({}, dict(softcap=-2.0), INV), ({}, dict(slopes=at(7) + 2), INV), (dict(S=0), {}, la.LA_OK)])
def test_swa_step_refusals(lib, base, kw, status):
    assert lib.la_swa_biased_decode_step(ctypes.byref(swa_step_args(base, **kw)), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(y=T(at(1), 100, 0, 64)), INV), (dict(y=T(at(1), 64, 0, 64)), INV), (dict(y=T(at(1), 64, 0, 96)), INV),
    # time-major output: the sequences lie within a token's row; no pointer for the taps is the next thing to refuse
    (dict(y=T(at(1), 64, 0, 128), w=None), INV)])
def test_conv_output_must_not_overlap_itself(lib, kw, status):
    assert lib.la_conv_prefill(ctypes.byref(conv_args(**kw)), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(o=T(at(3), 5120, 640, 64)), INV), (dict(o=T(at(3), 64, 1280, 64)), INV), (dict(softcap=2e37), INV), (dict(softcap=1e-39), INV),
    (dict(softcap=30.0, scale=float("inf")), INV), (dict(softcap=30.0, scale=float("nan")), INV),
    # one query of each of 2^31 heads: more rows than a launch's grid counts
    (dict(B=1 << 20, H=1 << 11, H_kv=1, Nq=1, Nk=1, k_cache=None, v_cache=None), UNS),
    (dict(B=1 << 20, H_kv=4, H=4, window=256 * 16, k_cache=None, v_cache=None, o=T(at(3), 0, 1280, 64)), INV)])
def test_swa_prefill_refuses_overlapping_outputs_extreme_caps_and_counts(lib, kw, status):
    assert lib.la_swa_prefill(ctypes.byref(swa_args(**kw)), None) == status


def test_swa_step_refuses_extreme_caps(lib):
    assert lib.la_swa_biased_decode_step(ctypes.byref(swa_step_args(softcap=1e-39)), None) == INV
    assert lib.la_swa_biased_decode_step(ctypes.byref(swa_step_args(softcap=1e38)), None) == INV


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_swa_prefill_refuses_bf16_strides_that_no_tensor_map_holds(lib, name):
    far = T(at(1), 1 << 39, 1280, 64)
    assert lib.la_swa_prefill(ctypes.byref(swa_args(**{name: far})), None) == UNS
    # fp32 inputs take any stride: their misaligned slopes are the next thing to refuse
    fp32 = dict(in_dtype=la.LA_DTYPE_F32, slopes=at(4) + 1)
    assert lib.la_swa_prefill(ctypes.byref(swa_args(**{name: far}, **fp32)), None) == INV


def test_counts_beyond_a_launchs_grid_are_refused(lib):
    """One short sequence too many for the launch that fills the padding, or for the convolution's own."""
    for B, N, status in ((1 << 31, 1, UNS), ((1 << 32) + 5, 1, UNS), (1 << 31, 0, UNS), ((1 << 32) + 5, 64, UNS), ((1 << 31) - 1, 1, INV)):
        wide = lambda k: T(at(k), 8 * max(N, 1), 0, 8)  # noqa: E731
        kw = dict(B=B, N=N, C=1, x=wide(0), y=wide(1), lens=at(6), fill=3)
        # within the limits the missing taps are the next thing to refuse
        assert lib.la_conv_prefill(ctypes.byref(conv_args(w=None, **kw)), None) == status
    assert lib.la_conv_prefill(ctypes.byref(conv_args(B=1 << 20, N=1 << 19, C=1, x=T(at(0), 1 << 22, 0, 8), y=T(at(1), 1 << 22, 0, 8))), None) == UNS
    for S, status in ((1 << 39, UNS), ((1 << 39) - 256, INV)):
        assert lib.la_conv_decode_step(ctypes.byref(conv_step_args(S=S, C=1, x_stride=8, out_stride=8, w=None)), None) == status
    B, N = 65535, 1 << 29
    big = dict(B=B, N=N, C=1, G=1, u=T(at(0), 0, 0, 8), delta=T(at(1), 0, 0, 8), z=T(None, 0, 0, 0), y=T(at(3), 8 * N, 0, 8),
               Bm=T(at(4), 0, 0, 16), Cm=T(at(5), 0, 0, 16), A=None)
    assert lib.la_ssm_prefill(ctypes.byref(ssm_args(**big)), None, 0, None) == UNS


def test_null_arguments(lib):
    for fn in (lib.la_conv_prefill, lib.la_conv_decode_step, lib.la_ssm_decode_step, lib.la_swa_prefill, lib.la_swa_biased_decode_step):
        assert fn(None, None) == INV
    assert lib.la_ssm_prefill(None, None, 0, None) == INV


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    x = torch.zeros((1, 4, 8))
    with pytest.raises(ValueError):
        la.la_conv_prefill(x, torch.zeros((8, 4)))
    with pytest.raises(ValueError):
        la.la_ssm_prefill(x, x, torch.zeros((8, 4)), torch.zeros((1, 1, 4, 4)), torch.zeros((1, 1, 4, 4)))
    with pytest.raises(ValueError):
        la.la_swa_prefill(torch.zeros((1, 2, 4, 8)), torch.zeros((1, 2, 4, 8)), torch.zeros((1, 2, 4, 8)))
    t = torch.zeros((2, 4))
    for bad in (("t", t, (1, 4), torch.float32, True), ("t", t, (2, 4), torch.bfloat16, True), ("t", t, (2, 4), torch.float32, True)):
        with pytest.raises(ValueError):
            la._check(t.get_device(), bad)  # a host tensor's index is -1: refused whatever its shape
    with pytest.raises(ValueError):
        la._refuse(-1, *("t", t, (2, 4), torch.float32, True))


def test_packed_arguments_are_the_structures_bytes():
    """The binding packs each argument struct in one call: the same bytes as the ctypes structure of the header."""
    T4 = lambda k: T(at(k), 1 + k, 2 + k, 3 + k)  # noqa: E731
    W4 = lambda k: (at(k), 1 + k, 2 + k, 3 + k)  # noqa: E731
    cases = [
        (la._CONV_PREFILL, la.ConvPrefillArgs(1, 2, 3, 4, 1, 0, 1, T4(0), T4(1), at(2), at(3), at(4), at(5), at(6), 1, 3),
         (1, 2, 3, 4, 1, 0, 1, *W4(0), *W4(1), at(2), at(3), at(4), at(5), at(6), 1, 3)),
        (la._CONV_DECODE, la.ConvDecodeArgs(1, 2, 3, 1, 0, 1, at(0), 5, at(1), 6, at(2), at(3), at(4), at(5), 1),
         (1, 2, 3, 1, 0, 1, at(0), 5, at(1), 6, at(2), at(3), at(4), at(5), 1)),
        (la._SSM_PREFILL, la.SsmPrefillArgs(1, 2, 3, 4, 5, 1, 0, *(T4(k) for k in range(6)), *(at(k) for k in range(6, 12)), 1, 2),
         (1, 2, 3, 4, 5, 1, 0, *(w for k in range(6) for w in W4(k)), *(at(k) for k in range(6, 12)), 1, 2)),
        (la._SSM_DECODE, la.SsmDecodeArgs(1, 2, 3, 4, 1, 0, *(T4(k) for k in range(6)), *(at(k) for k in range(6, 11)), 1),
         (1, 2, 3, 4, 1, 0, *(w for k in range(6) for w in W4(k)), *(at(k) for k in range(6, 11)), 1)),
        (la._SWA_PREFILL, la.SwaPrefillArgs(1, 2, 3, 4, 5, 6, 7, 1, 0, *(T4(k) for k in range(4)), 0.5, 2.5, at(4), at(5), at(6), 9, at(7),
                                            at(8), at(9), 1),
         (1, 2, 3, 4, 5, 6, 7, 1, 0, *(w for k in range(4) for w in W4(k)), 0.5, 2.5, at(4), at(5), at(6), 9, at(7), at(8), at(9), 1)),
        (la._SWA_BIASED_DECODE, la.SwaBiasedDecodeArgs(la.SwaDecodeArgs(1, 2, 3, 4, 1, 0, *(at(k) for k in range(7)), 0.5), 8, 1.5, at(9)),
         (1, 2, 3, 4, 1, 0, *(at(k) for k in range(7)), 0.5, 8, 1.5, at(9))),
    ]
    for packer, struct, words in cases:
        assert packer.size == ctypes.sizeof(struct)
        assert packer.pack(*words) == bytes(struct)
