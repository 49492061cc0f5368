"""Host-side checks of the linear attention and group norm calls: refusals with nothing launched."""
import ctypes

import pytest
import torch

import gated_delta_rule_31_gb300 as gdr
from gated_delta_rule_31_gb300 import LinearProblem, NormProblem

OK, INVALID, UNSUPPORTED, WORKSPACE = range(4)
FAKE, MISALIGNED = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100004)
ODD = ctypes.c_void_p(0x100001)
BIG = ctypes.c_size_t(1 << 60)


@pytest.fixture(scope="module")
def L():
    gdr.build()
    return gdr.lib()


def prob(**kw):
    base = dict(B=1, T=64, Hk=2, Hv=4, Dk=128, Dv=128, dtype=1, scale=0.1)
    base.update(kw)
    return LinearProblem(*[base[f] for f, _ in LinearProblem._fields_])


def norm(**kw):
    base = dict(rows=4, groups=2, D=64, dtype=1, activation=1, center=1, eps=1e-5)
    base.update(kw)
    return NormProblem(*[base[f] for f, _ in NormProblem._fields_])


def put(n, **at):
    """n fake pointers, some of them replaced (p3=None: the fourth is null)."""
    ptrs = [FAKE] * n
    for k, v in at.items():
        ptrs[int(k[1:])] = v
    return ptrs


@pytest.mark.parametrize("kw,code", [
    (dict(Hv=3), INVALID), (dict(Hk=0), INVALID), (dict(T=-1), INVALID), (dict(B=-2), INVALID), (dict(dtype=7), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(Dk=96), UNSUPPORTED),
    (dict(Dv=256), UNSUPPORTED), (dict(Dk=0), INVALID), (dict(B=70000), UNSUPPORTED), (dict(Hk=1, Hv=70000), UNSUPPORTED)])
def test_linear_problem(L, kw, code):
    p = ctypes.byref(prob(**kw))
    assert L.gdr_linear_fwd(p, *put(8), FAKE, BIG, None) == code
    assert L.gdr_linear_bwd(p, *put(12), FAKE, BIG, None) == code
    assert L.gdr_linear_fwd_workspace(p) == 0 and L.gdr_linear_bwd_workspace(p) == 0
    step = dict(kw, **({} if "T" in kw else {"T": 1}))
    assert L.gdr_linear_decode_step(ctypes.byref(prob(**step)), *put(6), None) == code


def test_linear_pointers(L):
    p = ctypes.byref(prob())
    assert L.gdr_linear_fwd(None, *put(8), FAKE, BIG, None) == INVALID
    for i in (0, 1, 2, 3, 6):  # q, k, v, g, o
        assert L.gdr_linear_fwd(p, *put(8, **{f"p{i}": None}), FAKE, BIG, None) == INVALID, i
    for i in (0, 1, 2, 4, 6, 7):  # 16-byte aligned ones
        assert L.gdr_linear_fwd(p, *put(8, **{f"p{i}": MISALIGNED}), FAKE, BIG, None) == INVALID, i
    for i in (3, 5):  # g, lengths
        assert L.gdr_linear_fwd(p, *put(8, **{f"p{i}": ODD}), FAKE, BIG, None) == INVALID, i
    for i in (0, 1, 2, 3, 6, 8, 9, 10):  # q, k, v, g, do, dq, dk, dv
        assert L.gdr_linear_bwd(p, *put(12, **{f"p{i}": None}), FAKE, BIG, None) == INVALID, i
    for i in (4, 6, 7, 8, 11):
        assert L.gdr_linear_bwd(p, *put(12, **{f"p{i}": MISALIGNED}), FAKE, BIG, None) == INVALID, i
    one = ctypes.byref(prob(T=1))
    for i in range(6):
        assert L.gdr_linear_decode_step(one, *put(6, **{f"p{i}": None}), None) == INVALID, i
    assert L.gdr_linear_decode_step(ctypes.byref(prob(T=2)), *put(6), None) == INVALID


def test_linear_workspace(L):
    for f, n in ((L.gdr_linear_fwd, 8), (L.gdr_linear_bwd, 12)):
        need = (L.gdr_linear_fwd_workspace if n == 8 else L.gdr_linear_bwd_workspace)(ctypes.byref(prob()))
        assert need > 0
        p = ctypes.byref(prob())
        assert f(p, *put(n), FAKE, ctypes.c_size_t(need - 1), None) == WORKSPACE
        assert f(p, *put(n), None, BIG, None) == WORKSPACE
        assert f(p, *put(n), ctypes.c_void_p(0x100010), BIG, None) == INVALID


def test_kept_states(L):
    p = ctypes.byref(prob(T=129))
    need = L.gdr_linear_states_bytes(p)
    assert need == 4 * 2 * 32768  # value heads x chunks of 128 tokens
    assert L.gdr_linear_states_bytes(ctypes.byref(prob(dtype=0))) == 0
    assert 0 < L.gdr_linear_bwd_states_workspace(p) < L.gdr_linear_bwd_workspace(p)
    assert L.gdr_linear_states_bytes(ctypes.byref(prob(Hv=3))) == 0

    def fwd(states, n):
        return L.gdr_linear_fwd_states(p, *put(8), states, ctypes.c_size_t(n), FAKE, BIG, None)

    def bwd(states, n):
        return L.gdr_linear_bwd_states(p, *put(6), states, ctypes.c_size_t(n), *put(6), FAKE, BIG, None)

    for f in (fwd, bwd):
        assert f(FAKE, need - 1) == WORKSPACE and f(None, need) == WORKSPACE
        assert f(ctypes.c_void_p(0x100010), need) == INVALID
    small = ctypes.c_size_t(L.gdr_linear_bwd_states_workspace(p) - 1)
    assert L.gdr_linear_bwd_states(p, *put(6), FAKE, BIG, *put(6), FAKE, small, None) == WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(groups=0), INVALID), (dict(D=0), INVALID), (dict(dtype=2), INVALID),
    (dict(activation=3), INVALID), (dict(center=2), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(D=8193), UNSUPPORTED), (dict(groups=1 << 20, D=64), UNSUPPORTED)])
def test_norm_problem(L, kw, code):
    p = ctypes.byref(norm(**kw))
    assert L.gdr_group_norm_fwd(p, *put(5), None) == code
    assert L.gdr_group_norm_bwd(p, *put(9), FAKE, BIG, None) == code
    assert L.gdr_group_norm_bwd_workspace(p) == 0


def test_norm_pointers_and_workspace(L):
    p = ctypes.byref(norm())
    assert L.gdr_group_norm_fwd(None, *put(5), None) == INVALID
    for i in (0, 4):  # x, y
        assert L.gdr_group_norm_fwd(p, *put(5, **{f"p{i}": None}), None) == INVALID
    for i in range(5):
        assert L.gdr_group_norm_fwd(p, *put(5, **{f"p{i}": ODD}), None) == INVALID, i
    for i in (0, 4, 5):  # x, dy, dx
        assert L.gdr_group_norm_bwd(p, *put(9, **{f"p{i}": None}), FAKE, BIG, None) == INVALID
    assert L.gdr_group_norm_bwd(p, *put(9, p1=None), FAKE, BIG, None) == INVALID  # dgate without a gate
    assert L.gdr_group_norm_bwd(p, *put(9, p6=None), FAKE, BIG, None) == INVALID  # a gate without dgate
    need = L.gdr_group_norm_bwd_workspace(p)
    assert need > 256
    assert L.gdr_group_norm_bwd(p, *put(9), FAKE, ctypes.c_size_t(need - 1), None) == WORKSPACE
    assert L.gdr_group_norm_bwd(p, *put(9), ctypes.c_void_p(0x100010), BIG, None) == INVALID


def test_binding_refuses():
    t = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        gdr.linear_fwd(t(1, 4, 1, 32), t(1, 4, 1, 32), t(1, 4, 1, 32), t(1))
    with pytest.raises(ValueError, match="CUDA"):
        gdr.linear_decode_step(t(1, 1, 32), t(1, 1, 32), t(1, 1, 32), t(1), t(1, 1, 32, 32))
    with pytest.raises(ValueError, match="CUDA"):
        gdr.group_norm_fwd(t(4, 64), 2)
    from gated_delta_rule_31_gb300.autograd import linear_attention

    with pytest.raises(ValueError, match="decay"):
        linear_attention(t(1, 4, 1, 32), t(1, 4, 1, 32), t(1, 4, 1, 32), t(1, requires_grad=True))


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu():
    dev = torch.device("cuda:0")
    q, v, g = torch.zeros(2, 8, 2, 64, device=dev), torch.zeros(2, 8, 4, 32, device=dev), torch.zeros(4, device=dev)
    ok = dict(q=q, k=q, v=v, g=g)

    def fwd(**kw):
        return gdr.linear_fwd(**{**ok, **kw})

    assert fwd()[0].shape == v.shape
    for kw in (dict(k=q[:, :7].contiguous()), dict(v=v[:1]), dict(g=g[:3]), dict(g=g.double()), dict(k=q.bfloat16()),
               dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(h0=torch.zeros(2, 4, 64, 32, device=dev)),
               dict(lengths=torch.zeros(2, dtype=torch.int64, device=dev)), dict(lengths=torch.zeros(3, dtype=torch.int32, device=dev)),
               dict(workspace=torch.empty(16, dtype=torch.uint8, device=dev)), dict(q=q.half(), k=q.half(), v=v.half()),
               dict(q=q[:, 0], k=q[:, 0])):
        with pytest.raises(ValueError):
            fwd(**kw)
    with pytest.raises(gdr.GdrError):
        fwd(scale=float("nan"))
    with pytest.raises(ValueError):
        gdr.linear_decode_step(q[:, 0].contiguous(), q[:, 0].contiguous(), v[:, 0].contiguous(), g, torch.zeros(2, 4, 64, 32, device=dev))
    x = torch.zeros(6, 64, device=dev)
    for args, kw in (((x, 3), {}), ((x, 0), {}), ((x.half(), 2), {}), ((x, 2, x[0].bfloat16()), {}), ((x, 2, None, x[0, :32]), {}),
                     ((x, 2, None, None, x[:5]), {}), ((x, 2), dict(activation="relu")), ((x.t(), 2), {})):
        with pytest.raises(ValueError):
            gdr.group_norm_fwd(*args, **kw)
    with pytest.raises(gdr.GdrError):
        gdr.group_norm_fwd(x, 2, eps=0.0)
    with pytest.raises(ValueError):
        gdr.group_norm_bwd(x, 2, None, None, None, x[:5])
