"""Host-side checks of the softmax attention layer's calls: refusals with nothing launched."""
import ctypes

import pytest

import gated_delta_rule_31_gb300 as gdr
from gated_delta_rule_31_gb300 import AppendProblem, PagedProblem, RotaryProblem, WindowProblem

OK, INVALID, UNSUPPORTED, WORKSPACE = range(4)
FAKE, MISALIGNED, ODD = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100004), ctypes.c_void_p(0x100001)
BIG = ctypes.c_size_t(1 << 60)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    gdr.build()
    return gdr.lib()


def make(cls, base, **kw):
    p = cls()
    for k, v in {**base, **kw}.items():
        setattr(p, k, (ctypes.c_int * 4)(*v) if k == "sections" else v)
    return ctypes.byref(p)


def window(**kw):
    return make(WindowProblem, dict(B=1, T=64, Hq=4, Hk=2, D=128, window=0, sinks=0, dtype=1, scale=0.1), **kw)


def rotary(**kw):
    return make(RotaryProblem, dict(B=1, T=64, H=4, D=128, pairs=64, axes=2, sections=(30, 34), interleaved=0, inverse=0, dtype=1), **kw)


def append(**kw):
    return make(AppendProblem, dict(B=1, T=4, Hq=4, Hk=2, D=128, pages=8, page_size=16, table_pages=3, pairs=64, axes=1, sections=(64,),
                                    interleaved=0, dtype=1), **kw)


def paged(**kw):
    return make(PagedProblem, dict(B=1, Hq=4, Hk=2, D=128, pages=8, page_size=16, table_pages=3, window=0, sinks=0, dtype=1, scale=0.1), **kw)


def put(n, **at):
    ptrs = [FAKE] * n
    for k, v in at.items():
        ptrs[int(k[1:])] = v
    return ptrs


HEADS = [(dict(Hq=3), INVALID), (dict(Hk=0), INVALID), (dict(Hq=0), INVALID), (dict(D=0), INVALID), (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
         (dict(B=-1), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(dtype=2), INVALID), (dict(scale=NAN), INVALID),
         (dict(scale=INF), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(B=70000), UNSUPPORTED),
         (dict(Hq=70000, Hk=1), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", HEADS + [(dict(T=-1), INVALID), (dict(T=(1 << 24) + 1), UNSUPPORTED),
                                             (dict(B=60000, T=1 << 24, Hq=64, Hk=64), UNSUPPORTED)])
def test_window_problem(L, kw, code):
    p = window(**kw)
    assert L.gdr_window_fwd(p, *put(7), FAKE, BIG, None) == code
    assert L.gdr_window_bwd(p, *put(11), FAKE, BIG, None) == code
    assert L.gdr_window_fwd_workspace(p) == 0 and L.gdr_window_bwd_workspace(p) == 0


def test_window_pointers(L):
    p = window()
    assert L.gdr_window_fwd(None, *put(7), FAKE, BIG, None) == INVALID
    assert L.gdr_window_fwd_workspace(None) == 0
    for i in (0, 1, 2, 4):  # q, k, v, o
        for bad in (None, MISALIGNED):
            assert L.gdr_window_fwd(p, *put(7, **{f"p{i}": bad}), FAKE, BIG, None) == INVALID, i
    for i in (3, 5):  # lengths, lse
        assert L.gdr_window_fwd(p, *put(7, **{f"p{i}": ODD}), FAKE, BIG, None) == INVALID, i
    assert L.gdr_window_fwd(p, *put(7, p6=MISALIGNED), FAKE, BIG, None) == INVALID  # rest
    assert L.gdr_window_bwd(p, *put(11, p6=MISALIGNED), FAKE, BIG, None) == INVALID
    assert L.gdr_window_fwd(window(dtype=0), *put(7), FAKE, BIG, None) == INVALID  # of bf16 only
    assert L.gdr_window_bwd(window(dtype=0), *put(11), FAKE, BIG, None) == INVALID
    for i in (0, 1, 2, 4, 7, 8, 9, 10):  # q, k, v, o, do, dq, dk, dv
        for bad in (None, MISALIGNED):
            assert L.gdr_window_bwd(p, *put(11, **{f"p{i}": bad}), FAKE, BIG, None) == INVALID, i
    assert L.gdr_window_bwd(p, *put(11, p5=None), FAKE, BIG, None) == INVALID  # lse
    for f, n, need in ((L.gdr_window_fwd, 7, L.gdr_window_fwd_workspace(p)), (L.gdr_window_bwd, 11, L.gdr_window_bwd_workspace(p))):
        assert need > 0
        assert f(p, *put(n), FAKE, ctypes.c_size_t(need - 1), None) == WORKSPACE
        assert f(p, *put(n), None, BIG, None) == WORKSPACE
        assert f(p, *put(n), MISALIGNED, BIG, None) == INVALID


TURN = [(dict(D=0), INVALID), (dict(D=127, pairs=20, axes=1, sections=(20,)), UNSUPPORTED), (dict(pairs=65, axes=1, sections=(65,)), INVALID),
        (dict(pairs=-1), INVALID), (dict(axes=0), INVALID), (dict(axes=5), INVALID), (dict(sections=(64, 1), axes=2), INVALID),
        (dict(sections=(65, -1), axes=2), INVALID), (dict(sections=(2 ** 31 - 1,) * 4, axes=4), INVALID), (dict(interleaved=2), INVALID),
        (dict(dtype=5), INVALID), (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(B=65536, T=65536), UNSUPPORTED),
        (dict(D=1 << 17), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", TURN + [(dict(H=0), INVALID), (dict(H=70000), UNSUPPORTED), (dict(inverse=-1), INVALID)])
def test_rotary_problem(L, kw, code):
    assert L.gdr_rotary(rotary(**kw), *put(4), None) == code


def test_rotary_pointers(L):
    assert L.gdr_rotary(None, *put(4), None) == INVALID
    for i in range(4):  # x, positions, inv_freq, y
        for bad in (None, ODD):
            assert L.gdr_rotary(rotary(), *put(4, **{f"p{i}": bad}), None) == INVALID, i
    assert L.gdr_rotary(rotary(T=0), *put(4, p0=None, p1=None, p2=None, p3=None), None) == OK
    assert L.gdr_rotary(rotary(dtype=0), *put(4, p0=ctypes.c_void_p(0x100002)), None) == INVALID


@pytest.mark.parametrize("kw,code", TURN + [(dict(Hq=-1), INVALID), (dict(Hk=0), INVALID), (dict(Hq=70000), UNSUPPORTED), (dict(Hk=70000), UNSUPPORTED),
                                            (dict(pages=-1), INVALID), (dict(page_size=0), INVALID), (dict(table_pages=-1), INVALID)])
def test_append_problem(L, kw, code):
    assert L.gdr_kv_append(append(**kw), *put(11), None) == code


def test_append_pointers(L):
    assert L.gdr_kv_append(None, *put(11), None) == INVALID
    for i in (0, 1, 2, 4, 5, 7, 8, 9, 10):  # q, k, v, inv_freq, lengths, page_table, q_out, caches
        for bad in (None, ODD):
            assert L.gdr_kv_append(append(), *put(11, **{f"p{i}": bad}), None) == INVALID, i
    for i in (3, 6):  # positions, counts
        assert L.gdr_kv_append(append(), *put(11, **{f"p{i}": ODD}), None) == INVALID, i
    # several axes need positions
    assert L.gdr_kv_append(append(axes=2, sections=(32, 32)), *put(11, p3=None), None) == INVALID
    assert L.gdr_kv_append(append(B=0), *[None] * 11, None) == OK
    assert L.gdr_kv_append(append(Hq=0, pages=0), *put(11, p0=None, p8=None, p9=None, p10=None), None) == OK  # nowhere to write


@pytest.mark.parametrize("kw,code", HEADS + [(dict(pages=-1), INVALID), (dict(page_size=0), INVALID), (dict(table_pages=-1), INVALID),
                                             (dict(pages=1 << 20, page_size=1 << 12), UNSUPPORTED),
                                             (dict(table_pages=1 << 27), UNSUPPORTED)])
def test_paged_problem(L, kw, code):
    p = paged(**kw)
    assert L.gdr_paged_decode_step(p, *put(6), FAKE, BIG, None) == code
    assert L.gdr_paged_decode_workspace(p) == 0


def test_paged_pointers(L):
    p = paged()
    assert L.gdr_paged_decode_step(None, *put(6), FAKE, BIG, None) == INVALID
    for i in (0, 1, 2, 5):  # q, caches, o
        for bad in (None, MISALIGNED):
            assert L.gdr_paged_decode_step(p, *put(6, **{f"p{i}": bad}), FAKE, BIG, None) == INVALID, i
    for i in (3, 4):  # page_table, lengths
        for bad in (None, ODD):
            assert L.gdr_paged_decode_step(p, *put(6, **{f"p{i}": bad}), FAKE, BIG, None) == INVALID, i
    need = L.gdr_paged_decode_workspace(p)
    assert L.gdr_paged_decode_step(p, *put(6), FAKE, ctypes.c_size_t(need - 1), None) == WORKSPACE
    assert L.gdr_paged_decode_step(p, *put(6), MISALIGNED, BIG, None) == INVALID
    assert L.gdr_paged_decode_step(paged(B=0), *[None] * 5, None, FAKE, BIG, None) == OK
