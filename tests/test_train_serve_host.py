"""Refusals of the balance loss, the AdamW step and the adapters of many requests, on the host
before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

import mixture_experts_lora_b200 as ml

P = ctypes.c_void_p
FAKE, ODD = P(4096), P(4100)       # never dereferenced


@pytest.fixture(scope="module")
def L():
    from mixture_experts_lora_b200 import build
    build.build(quiet=True)
    return ml.lib()


def test_balance_workspace(L):
    assert ml.moe_balance_workspace_bytes(4096, 128) > 0
    assert ml.moe_balance_workspace_bytes(0, 8) > 0
    assert ml.moe_balance_workspace_bytes(4096, 128, 64) > ml.moe_balance_workspace_bytes(4096, 128)
    for bad in ((-1, 8, 1), (4, 0, 1), (4, 1025, 1), (4, 8, 0), (4, 8, 1 << 24), (1 << 31, 8, 1)):
        assert ml.moe_balance_workspace_bytes(*bad) == 0


def test_balance_loss_refusals(L):
    def call(T=4, E=8, k=2, off=None, S=1, logits=FAKE, ids=FAKE, loss=FAKE, ws=FAKE, wsb=1 << 30):
        return L.moe_balance_loss(logits, ids, T, E, k, off, S, None, loss, FAKE, FAKE, ws, wsb, None)
    assert call(k=0) == call(E=1) == call(k=33, E=64) == call(E=1025) == ml.MOE_ERR_UNSUPPORTED
    assert call(T=1 << 30, k=2) == call(S=1 << 24, off=FAKE) == ml.MOE_ERR_UNSUPPORTED
    assert call(T=-1) == call(S=0) == call(S=2) == ml.MOE_ERR_INVALID_ARG      # S = 2 needs offsets
    assert call(logits=None) == call(ids=None) == call(loss=None) == call(ws=None) == ml.MOE_ERR_INVALID_ARG
    assert call(ws=ODD) == ml.MOE_ERR_INVALID_ARG
    assert call(wsb=ml.moe_balance_workspace_bytes(4, 8) - 1) == ml.MOE_ERR_WORKSPACE


def test_balance_backward_refusals(L):
    def call(T=4, E=8, k=2, off=None, S=1, logits=FAKE, counts=FAKE, dloss=FAKE, out=FAKE):
        return L.moe_balance_loss_backward(logits, counts, FAKE, dloss, T, E, k, off, S, None, out, 0, None)
    assert call(k=0) == call(E=1) == call(E=1025) == ml.MOE_ERR_UNSUPPORTED
    assert call(T=-1) == call(S=2) == call(logits=None) == call(counts=None) == ml.MOE_ERR_INVALID_ARG
    assert call(dloss=None) == call(out=None) == ml.MOE_ERR_INVALID_ARG
    assert call(T=0, out=None) == ml.MOE_OK


def _adamw(L, step=FAKE, n=1, table=True, **kw):
    cfg = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, param_bf16=1, grad_bf16=1, has_master=0,
               state_bits=32)
    row = dict(param=4096, grad=4096, exp_avg=4096, exp_avg_sq=4096, exp_avg_scale=None, exp_avg_sq_scale=None,
               master=None, size=(1, 1, 64), param_stride=(0, 0, 1), grad_stride=(0, 0, 1))
    for k, v in kw.items():
        (cfg if k in cfg else row)[k] = v
    c = ml.moe_adamw_config_t(**cfg)
    t = (ml.moe_adamw_tensor_t * 1)()
    for k, v in row.items():
        if isinstance(v, tuple):
            getattr(t[0], k)[:] = v
        else:
            setattr(t[0], k, v)
    return L.moe_adamw_step(t if table else None, n, ctypes.byref(c), None, None, step, 1, None)


def test_adamw_refusals(L):
    bad = ml.MOE_ERR_INVALID_ARG
    assert _adamw(L, n=-1) == _adamw(L, table=False) == _adamw(L, step=None) == _adamw(L, step=ODD) == bad
    assert L.moe_adamw_step(None, 0, None, None, None, FAKE, 1, None) == bad
    for kw in (dict(lr=float("nan")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.5), dict(eps=-1.0),
               dict(eps=float("inf")), dict(weight_decay=float("inf")), dict(param=None), dict(grad=None),
               dict(param=4097), dict(exp_avg=None), dict(exp_avg_sq=4100), dict(size=(1, 1, -1)),
               dict(param_stride=(0, 0, -1)), dict(param_stride=(0, 0, 0)), dict(state_bits=8),
               dict(has_master=1), dict(has_master=1, master=4100),
               dict(param_bf16=0, param=4098), dict(grad_bf16=0, grad=4098)):
        assert _adamw(L, **kw) == bad, kw
    for kw in (dict(state_bits=16), dict(param_bf16=0, has_master=1, master=4096), dict(size=(1, 1, 1 << 41)),
               dict(size=(1 << 16, 1, 1 << 16), param_stride=(1 << 17, 0, 1))):
        assert _adamw(L, **kw) == ml.MOE_ERR_UNSUPPORTED, kw


def test_lora_requests_refusals(L):
    def call(X=FAKE, ldx=64, off=None, ad=FAKE, T=4, S=4, A=FAKE, B=FAKE, c=FAKE, n=2, K=64, N=32, r=8, Y=FAKE, ldy=32):
        return L.moe_lora_requests(X, ldx, off, ad, T, S, A, B, c, n, K, N, r, Y, ldy, None)
    assert call(K=40) == call(K=0) == call(N=24) == call(r=12) == call(r=136) == call(r=0) == ml.MOE_ERR_UNSUPPORTED
    assert call(T=1 << 24, S=1 << 24) == call(K=1 << 20, ldx=1 << 20) == ml.MOE_ERR_UNSUPPORTED
    for kw in (dict(T=-1), dict(S=-1), dict(n=-1), dict(S=3), dict(ldx=56), dict(ldx=68), dict(ldy=24), dict(X=None),
               dict(X=ODD), dict(Y=None), dict(Y=ODD), dict(ad=None), dict(A=None), dict(B=ODD), dict(c=None)):
        assert call(**kw) == ml.MOE_ERR_INVALID_ARG, kw
    assert call(T=0, S=0, X=None, Y=None) == ml.MOE_OK


def test_lora_requests_refuses_rows_that_overlap(L):
    def call(x, ldx, y, ldy, T=8, K=64, N=32):
        return L.moe_lora_requests(P(x), ldx, None, FAKE, T, T, FAKE, FAKE, FAKE, 2, K, N, 8, P(y), ldy, None)
    at = 1 << 20
    for y, ldx, ldy in ((at, 64, 64), (at + 112, 64, 64), (at - 16, 64, 32), (at + 2 * (7 * 64 + 56), 64, 32),
                        (at + 2 * 40, 96, 96), (at + 2 * 72, 96, 96), (at - 2 * 24, 96, 96), (at + 2 * (7 * 96 + 56), 96, 96),
                        (at + 2 * 64, 96, 104), (at - 2 * 7 * 96, 96, 96)):
        assert call(at, ldx, y, ldy) == ml.MOE_ERR_INVALID_ARG, (y - at, ldx, ldy)
    assert call(at, 64, at + 2 * 56, 32, T=1) == call(at, 64, at - 2 * 24, 32, T=1) == ml.MOE_ERR_INVALID_ARG


def test_bindings_refuse_cpu_tensors_and_wrong_types():
    z, i = torch.zeros, torch.int32
    with pytest.raises(ValueError):
        ml.moe_balance_loss(z(4, 8), z(4, 2, dtype=i), z(1), z(1, 8, dtype=i), z(1, dtype=i), z(1024))
    with pytest.raises(ValueError):
        ml.moe_balance_loss(z(4, 8).half(), z(4, 2, dtype=i), z(1), z(1, 8, dtype=i), z(1, dtype=i), z(1024))
    with pytest.raises(ValueError):
        ml.moe_balance_loss_backward(z(4, 8), z(1, 8, dtype=i), z(1, dtype=i), z(2), 2, z(4, 8))
    b = torch.bfloat16
    with pytest.raises(ValueError):
        ml.moe_lora_requests(z(4, 64, dtype=b), z(4, dtype=i), z(2, 64, 8, dtype=b), z(2, 8, 32, dtype=b), z(2),
                             z(4, 32, dtype=b))
    with pytest.raises(ValueError):
        ml.moe_lora_requests(z(4, 64), z(4, dtype=i), z(2, 64, 8, dtype=b), z(2, 8, 32, dtype=b), z(2), z(4, 32))
    with pytest.raises(ValueError):
        ml.AdamW([z(4)], [z(4)])
    with pytest.raises(ValueError):
        ml.AdamW([], [])
    with pytest.raises(ValueError):
        ml.AdamW([z(4)], [z(4)], state_bits=4)


@pytest.mark.parametrize("E", [3, 64, 128, 256, 257, 1024])
@pytest.mark.parametrize("S", [1, 4, 5, 29, 295, 296, 297, 5000])
def test_a_balance_workspace_for_a_batch_does_for_shorter_ones(L, E, S):
    rows = sorted({*range(0, 400), *range(400, 140000, 97), *(32 * b + d for b in range(1, 4400) for d in (-1, 0, 1)),
                   18944, 18945, 130832, 131072, (1 << 31) - 1})
    need = [ml.moe_balance_workspace_bytes(T, E, S) for T in rows]
    assert all(a <= b for a, b in zip(need, need[1:]))
    # nor does a sequence more need less
    assert all(ml.moe_balance_workspace_bytes(T, E, S) <= ml.moe_balance_workspace_bytes(T, E, S + 1)
               for T in (0, 1, 40, 1024, 1025, 9000, 18944, 18945, 131071, 1 << 24))


def test_adamw_refuses_views_whose_elements_meet(L):
    for size, stride in (((1, 8, 8), (0, 4, 1)), ((1, 8, 8), (0, 1, 4)), ((9, 8, 8), (8, 64, 1)), ((2, 2, 2), (0, 2, 1)),
                         ((2, 1, 8), (7, 0, 1)), ((3, 1 << 20, 2), (1 << 20, 2, 1))):
        assert _adamw(L, size=size, param_stride=stride, grad_stride=stride) == ml.MOE_ERR_INVALID_ARG, (size, stride)


@pytest.mark.parametrize("eps", [1e-39, 1e-50, 2.0 ** -127])
def test_adamw_refuses_an_eps_below_the_normal_numbers(L, eps):
    assert _adamw(L, eps=eps) == ml.MOE_ERR_INVALID_ARG
