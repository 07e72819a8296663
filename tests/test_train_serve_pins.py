"""Pins of the fp64 definitions in oracle/train_serve_oracle.py: differences, brute force,
torch's own AdamW, and planted mistakes (CPU)."""
import numpy as np
import pytest
import torch

import mixture_experts_lora_b200 as ml
import oracle.train_serve_oracle as O


def _routed(T=23, E=7, k=3, seed=0):
    g = np.random.default_rng(seed)
    logits = g.normal(size=(T, E))
    ids = np.argsort(-logits, axis=1)[:, :k]
    return logits, ids


def test_balance_loss_of_even_and_collapsed_routing():
    E, k = 8, 2
    T = 16
    ids = np.stack([(np.arange(T) * k + j) % E for j in range(k)], axis=1)
    loss, counts, n = O.balance_loss(np.zeros((T, E)), ids)
    assert np.allclose(loss, 1.0) and np.all(counts == T * k // E) and n[0] == T
    one = np.full((T, E), -40.0)
    one[:, 3] = 40.0
    assert np.isclose(O.balance_loss(one, np.full((T, 1), 3))[0][0], E)   # all on one expert


@pytest.mark.parametrize("masked", [False, True])
def test_balance_gradient_matches_differences(masked):
    logits, ids = _routed()
    off = [0, 9, 9, 20]                      # an empty sequence, rows behind the last one
    mask = (np.arange(23) % 4 != 1) if masked else None
    dloss = np.array([0.7, 1.3, -0.4])
    loss, counts, n = O.balance_loss(logits, ids, 3, off, mask)
    grad = O.balance_backward(logits, counts, n, dloss, 3, off, mask)
    h = 1e-6
    for t, e in [(0, 0), (1, 2), (4, 6), (9, 1), (19, 5), (20, 0), (22, 3)]:
        d = np.zeros_like(logits)
        d[t, e] = h
        up, dn = (np.sum(dloss * O.balance_loss(logits + x, ids, 3, off, mask)[0]) for x in (d, -d))
        assert abs((up - dn) / (2 * h) - grad[t, e]) < 1e-8
    assert not grad[20:].any() and loss[1] == 0
    wrong = O.balance_backward(logits, counts, n + 1, dloss, 3)      # a mistake shows
    assert np.abs(wrong - grad).max() > 1e-3


def test_adamw_matches_torch():
    g = np.random.default_rng(1)
    w0 = g.normal(size=50)
    p = torch.nn.Parameter(torch.tensor(w0))
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    w, m, v = w0.copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        grad = g.normal(size=50)
        p.grad = torch.tensor(grad)
        opt.step()
        w, m, v = O.adamw(w, grad, m, v, t, 3e-3, 0.8, 0.95, 1e-6, 0.1)
    assert np.allclose(w, p.detach().numpy(), rtol=1e-12, atol=0)


def test_e4m3_values_are_torchs():
    t = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, O.e4m3_values())


def test_codes_keep_the_mean_and_the_bounds():
    g = np.random.default_rng(2)
    x = g.normal(size=512) * np.exp(g.normal(size=512) * 2)
    steps = 4000
    mean = np.zeros(512)
    for t in range(1, steps + 1):
        codes, scales, _ = O.encode(x, O.noise(t, 512)[0])
        mean += O.decode(codes, scales) / steps
    top = np.repeat(np.abs(x.reshape(-1, 256)).max(axis=1), 256)
    gap = np.maximum(np.abs(x) / 8, top / 448 * 2.0 ** -9)      # a code is at most this wide
    # the mean of `steps` roundings has a deviation of at most gap / 2 / sqrt(steps)
    assert np.all(np.abs(mean - x) < 5 * gap / 2 / np.sqrt(steps) + gap * 2.0 ** -15)
    # rounding to nearest would keep a slowly falling value where it is; this follows it
    u = np.full(256, 0.5)
    u[0] = 1.0
    codes, scales, _ = O.encode(u, np.zeros(256), True)
    for t in range(1, 1001):
        u = O.decode(codes, scales) * 0.9995
        u[0] = 1.0
        codes, scales, _ = O.encode(u, O.noise(t, 256)[1], True)
    # 255 values, each after many roundings: deviation of the mean below 0.02
    assert abs(O.decode(codes, scales)[1:].mean() - 0.5 * 0.9995 ** 1000) < 0.06


def test_lora_requests_is_the_merged_weight():
    g = np.random.default_rng(3)
    X, W = g.normal(size=(9, 6)), g.normal(size=(6, 5))
    A, B, c = g.normal(size=(2, 6, 3)), g.normal(size=(2, 3, 5)), np.array([0.5, 2.0])
    off, ad = [0, 2, 2, 7], [1, 0, -1]
    Y = O.lora_requests(X, ad, A, B, c, X @ W, off)
    want = X @ W
    want[:2] = X[:2] @ (W + c[1] * A[1] @ B[1])
    assert np.allclose(Y, want)
    single = O.lora_requests(X, [0, 1, -1] * 3, A, B, c, X @ W)
    assert np.allclose(single[1], X[1] @ (W + c[1] * A[1] @ B[1])) and np.allclose(single[2], (X @ W)[2])


def test_joint_view_of_strided_tensors():
    def same(p, g):
        v = ml._joint_view(p, g)
        idx = np.indices([n for n, _, _ in v]).reshape(3, -1)
        for t, col in ((p, 1), (g, 2)):
            at = sum(i * x[col] for i, x in zip(idx, v))
            flat = torch.as_strided(t, (t.untyped_storage().nbytes() // t.element_size() - t.storage_offset(),), (1,))
            assert torch.equal(flat[torch.from_numpy(np.asarray(at).ravel()).long()], t.reshape(-1))
    x = torch.arange(4 * 6 * 10.0).view(4, 6, 10)
    same(x, x + 1)
    same(x[:, :, :5], x[:, :, 5:])
    same(x[:, :3, 2:7], torch.arange(60.0).view(4, 3, 5))
    same(x.transpose(0, 2), x.transpose(0, 2).contiguous())
    same(x[:, :1, 3:4], x[:, 1:2, :1])
    same(x[0, 0, :1], x[1, 1, :1])
    assert [n for n, _, _ in ml._joint_view(x, x)] == [1, 1, 240]
    with pytest.raises(ValueError):
        y = torch.zeros(3, 4, 5, 6)[:, :2, :3, :5]
        ml._joint_view(y, y)
