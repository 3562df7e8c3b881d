"""The output head's losses on the host: the 64-bit reference against torch
autograd and differences, and every refusal that needs no device."""
import math

import pytest
import torch

import head_ref as ref
import moe_grouped_gemm_bf16_amd as mg
from moe_grouped_gemm_bf16_amd import _lib

L = _lib.LIB
OK, NUL, SHAPE, ALIGN, DEV = range(5)
A = 0x10000          # an aligned fake address, never dereferenced
BIG = 1 << 60


def _inputs(T, V, D, seed):
    g = torch.Generator().manual_seed(seed)
    return g, torch.randn(T, D, generator=g).double(), torch.randn(V, D, generator=g).double()


@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_reference_against_autograd(tau):
    T, V, D, k = 7, 30, 5, 4
    g, x, w = _inputs(T, V, D, 1)
    x.requires_grad_(), w.requires_grad_()
    up = torch.randn(T, generator=g).double()
    index = torch.rand(T, V, generator=g).argsort(1)[:, :k].int()
    index[2] = -1
    index[3, 1:] = -1
    index[4, 1] = index[4, 0]
    teacher = torch.randn(T, k, generator=g)
    teacher[5, 0] = -math.inf
    at, q, size = ref.entries(teacher=teacher, index=index, temperature=tau)
    p = torch.log_softmax(x @ w.T / tau, 1)
    want = torch.where(q > 0, torch.xlogy(q, q) - q * p.gather(1, at.clamp_min(0)), 0.0).sum(1)
    loss, lse, *_ = ref.forward(x.detach(), w.detach(), at, q, size, tau)
    assert torch.allclose(loss, want, atol=1e-12)
    (want * up).sum().backward()
    dx, dw, *_ = ref.backward(x.detach(), w.detach(), at, q, size, lse, up, temperature=tau)
    assert torch.allclose(dx, x.grad, atol=1e-12) and torch.allclose(dw, w.grad, atol=1e-12)


def test_reference_gradient_with_z_loss_against_differences():
    T, V, D = 5, 12, 3
    g, x, w = _inputs(T, V, D, 2)
    t = torch.tensor([0, 11, -100, 5, 5], dtype=torch.int32)
    e = ref.entries(targets=t)
    up, c = torch.randn(T, generator=g).double(), 0.1

    def value(x, w):
        loss, lse, *_ = ref.forward(x, w, *e)
        return float((loss * up).sum() + c * (lse ** 2).sum())

    _, lse, *_ = ref.forward(x, w, *e)
    dx, dw, *_ = ref.backward(x, w, *e, lse, up, up + 2 * c * lse)
    for m, d in ((x, dx), (w, dw)):
        for i in range(m.shape[0]):
            for j in range(m.shape[1]):
                old = float(m[i, j])
                m[i, j] = old + 1e-5
                hi = value(x, w)
                m[i, j] = old - 1e-5
                lo = value(x, w)
                m[i, j] = old
                assert abs((hi - lo) / 2e-5 - float(d[i, j])) < 1e-8


def _loss(x=A, w=A, t=A, T=4, V=9, D=16, first=0, loss=A, lse=A, logit=A, ws=A, n=BIG):
    return L.mg_head_loss(x, w, t, T, V, D, first, loss, lse, logit, ws, n, None)


def _loss_bwd(x=A, w=A, t=A, lse=A, dloss=A, dlse=None, T=4, V=9, D=16, first=0, dx=A, dw=A, ws=A, n=BIG):
    return L.mg_head_loss_bwd(x, w, t, lse, dloss, dlse, T, V, D, first, dx, dw, ws, n, None)


def _distill(x=A, w=A, te=A, bf=0, i=A, T=4, V=9, D=16, k=3, first=0, tau=1.0, loss=A, lse=A, logits=A, ws=A, n=BIG):
    return L.mg_head_distill(x, w, te, bf, i, T, V, D, k, first, tau, loss, lse, logits, ws, n, None)


def _distill_bwd(x=A, w=A, te=A, bf=0, i=A, lse=A, z=A, dloss=A, T=4, V=9, D=16, k=3, first=0, tau=1.0, dx=A, dw=A, ws=A, n=BIG):
    return L.mg_head_distill_bwd(x, w, te, bf, i, lse, z, dloss, T, V, D, k, first, tau, dx, dw, ws, n, None)


ALL = [_loss, _loss_bwd, _distill, _distill_bwd]


@pytest.mark.parametrize("call", ALL)
def test_sizes(call):
    for bad in (dict(T=-1), dict(T=(1 << 22) + 1), dict(V=0), dict(V=-1), dict(V=1 << 31), dict(D=0), dict(D=12), dict(D=-8),
                dict(D=(1 << 20) + 8), dict(first=-1), dict(first=(1 << 31) - 8), dict(T=1 << 22, V=1 << 20), dict(V=1 << 21, D=1 << 20),
                dict(n=0)):
        assert call(**bad) == SHAPE, bad
    k = 3 if call in (_distill, _distill_bwd) else 0
    need = L.mg_head_bwd_workspace(4, 9, 16, k) if call in (_loss_bwd, _distill_bwd) else L.mg_head_workspace(4, 9, 16)
    assert call(n=need - 1) == SHAPE and call(n=need) in (OK, DEV, 5)
    for ok in (dict(T=0), dict(T=0, x=None, t=None, ws=None, n=0) if call is _loss else dict(T=0)):
        assert call(**ok) in (OK, DEV), ok                    # (a gradient of no tokens still writes zeros)


@pytest.mark.parametrize("call", [_distill, _distill_bwd])
def test_entries_and_temperature(call):
    for bad in (dict(k=0), dict(k=-1), dict(k=257), dict(T=1 << 22, k=256, V=1 << 31), dict(tau=0.0), dict(tau=-1.0), dict(tau=math.nan),
                dict(tau=math.inf), dict(tau=1e-45), dict(tau=3.4e38)):
        assert call(**bad) == SHAPE, bad


def test_pointers():
    for call, need, low in ((_loss, ("x", "w", "t", "loss", "lse", "logit", "ws"), ("t", "loss", "lse", "logit")),
                            (_loss_bwd, ("x", "w", "t", "lse", "dloss", "ws"), ("t", "lse", "dloss", "dlse")),
                            (_distill, ("x", "w", "te", "i", "loss", "lse", "logits", "ws"), ("te", "i", "loss", "lse", "logits")),
                            (_distill_bwd, ("x", "w", "te", "i", "lse", "z", "dloss", "ws"), ("te", "i", "lse", "z", "dloss"))):
        for name in need:
            assert call(**{name: None}) == NUL, (call, name)
        for name in low:
            assert call(**{name: A + 2}) == ALIGN, (call, name)
        for name in ("x", "w", "ws") + (("dx", "dw") if call in (_loss_bwd, _distill_bwd) else ()):
            assert call(**{name: A + 8}) == ALIGN, (call, name)
    assert _distill(te=A + 1, bf=1) == ALIGN and _distill(te=A + 2, bf=1) == DEV       # 16-bit values
    for call in (_loss_bwd, _distill_bwd):
        assert call(dx=None, dw=None) == OK                    # nothing is wanted


def test_without_a_device():
    assert [c() for c in ALL] == [DEV] * 4 or torch.cuda.is_available()


def test_workspace_sizes():
    assert L.mg_head_workspace(0, 9, 16) == 0 and L.mg_head_workspace(4, 9, 12) == 0 and L.mg_head_workspace(4, 0, 16) == 0
    assert L.mg_head_bwd_workspace(4, 9, 16, 257) == 0 and L.mg_head_bwd_workspace(4, 9, 16, -1) == 0
    for T, V, D in ((1, 1, 8), (8192, 131072, 4096), (65536, 200000, 2048), (300, 100, 72)):
        fwd, bwd = L.mg_head_workspace(T, V, D), L.mg_head_bwd_workspace(T, V, D, 0)
        wide = -(-D // 64) * 64                       # packed rows of x start on 128 bytes
        # (up to 128 tokens: up to 256 tiles more, of four parts of 8 bytes; and a
        # tile of 256 entries more, 256 bytes for each of the parts)
        assert 0 < fwd < 2 * T * wide + 40 * T + V * T / 8 + (8192 * T if T <= 128 else 0) + 32 * T + 4096
        assert 0 < bwd < (1 << 30) + 8 * (T + 256) * wide + 40 * T + 4096
        # the entries' places and values are kept where the vocabulary goes in pieces
        assert L.mg_head_bwd_workspace(T, V, D, 64) >= bwd + (6 * 64 * T if T * V > 1 << 28 else 0)


def test_binding_refuses_before_any_launch():
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(9, 16, dtype=torch.bfloat16)
    t, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU device"):
        mg.head_loss(x, w, t)
    with pytest.raises(TypeError, match="bfloat16"):
        mg.head_loss(x.float(), w, t)
    with pytest.raises(ValueError, match="2 dims"):
        mg.head_loss(x[0], w, t)
    with pytest.raises(TypeError, match="Tensor"):
        mg.head_loss_bwd(x.numpy if False else None, w, t, f, f)
    with pytest.raises(ValueError, match="GPU device"):
        mg.head_distill_bwd(x, w, f[:, None], t[:, None], f, f[:, None], f)


@pytest.mark.gpu
def test_binding_refusals_with_a_device():
    d = "cuda"
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16, device=d), torch.zeros(9, 16, dtype=torch.bfloat16, device=d)
    t, f, i, te = torch.zeros(4, dtype=torch.int32, device=d), torch.zeros(4, device=d), torch.zeros(4, 3, dtype=torch.int32, device=d), torch.zeros(4, 3, device=d)
    for err, call in (
            (ValueError, lambda: mg.head_loss(x, w[:, :8].contiguous(), t)), (ValueError, lambda: mg.head_loss(x, w, t[:3])),
            (TypeError, lambda: mg.head_loss(x, w, t.long())), (ValueError, lambda: mg.head_loss(x.t(), w, t)),
            (ValueError, lambda: mg.head_loss(x, w, t, first=-1)), (ValueError, lambda: mg.head_loss(x, w, t, first=2 ** 31 - 8)),
            (ValueError, lambda: mg.head_loss(x, w, t.cpu())), (mg.MgemmError, lambda: mg.head_loss(x, w[:0], t)),
            (mg.MgemmError, lambda: mg.head_loss(x[:, :4].contiguous(), w[:, :4].contiguous(), t)),
            (ValueError, lambda: mg.head_loss_bwd(x, w, t, f[:3], f)), (ValueError, lambda: mg.head_loss_bwd(x, w, t, f, f, dlse=f[:2])),
            (TypeError, lambda: mg.head_loss_bwd(x, w, t, f.double(), f)), (ValueError, lambda: mg.head_loss_bwd(x, w, t, f, f, dx=w)),
            (ValueError, lambda: mg.head_loss_bwd(x, w, t, f, f, dw=w.clone(), need_dw=False)),
            (TypeError, lambda: mg.head_distill(x, w, te.half(), i)), (ValueError, lambda: mg.head_distill(x, w, te[:, :2].contiguous(), i)),
            (TypeError, lambda: mg.head_distill(x, w, te, i.long())), (ValueError, lambda: mg.head_distill(x, w, te, i, temperature=0.0)),
            (ValueError, lambda: mg.head_distill(x, w, te, i, temperature=math.nan)),
            (ValueError, lambda: mg.head_distill(x, w, te.expand(4, 3)[:, :0].contiguous(), i[:, :0].contiguous())),
            (ValueError, lambda: mg.head_distill_bwd(x, w, te, i, f, te[:, :2].contiguous(), f))):
        with pytest.raises(err):
            call()
