"""The operators as they are used together: the layer's training step (routing, balance loss,
backward, AdamW on its adapters), and the trained adapters served in one batch."""
import numpy as np
import pytest
import torch

import mixture_experts_lora_b200 as ml
import oracle.moe_lora_oracle as OL
import oracle.train_serve_oracle as O
from moe_inputs import generate, small_config

from gpu_common import TOL, ensure_built, inputs_on, rel_err, to_np

pytestmark = pytest.mark.gpu
ADAPTERS = ("A_gu", "B_gu", "A_d", "B_d")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


@pytest.mark.parametrize("bits,graph", [(32, False), (8, False), (32, True)])
def test_training_steps(bits, graph):
    cfg = small_config(T=200, m=128, n=64, E=8, k=2, r=8, alpha=16)
    inp, cpu = inputs_on(cfg)
    buf = ml.alloc_buffers(cfg.T, cfg.m, cfg.n, cfg.E, cfg.k, cfg.r, cfg.scale)
    bal = ml.alloc_balance(cfg.T, cfg.E, 2, weight=0.5)
    off = torch.tensor([0, 120, 190], dtype=torch.int32, device="cuda")
    opt = ml.AdamW([inp[n] for n in ADAPTERS], [buf.dA_gu, buf.dB_gu, buf.dA_d, buf.dB_d], lr=1e-3, state_bits=bits,
                   master_weights=True)
    step = lambda: ml.layer_train_step(inp, cfg.k, cfg.scale, buf, opt, bal, off)      # noqa: E731
    if graph:
        g = torch.cuda.CUDAGraph()
        # (the first call of every kernel outside the capture, on buffers of its own)
        warm, _ = inputs_on(cfg)
        wb = ml.alloc_buffers(cfg.T, cfg.m, cfg.n, cfg.E, cfg.k, cfg.r, cfg.scale)
        ml.layer_train_step(warm, cfg.k, cfg.scale, wb,
                            ml.AdamW([warm[n] for n in ADAPTERS], [wb.dA_gu, wb.dB_gu, wb.dA_d, wb.dB_d]))
        with torch.cuda.graph(g):
            step()
    for t in range(1, 4):
        master = [opt._part(opt.master, i).double().cpu().numpy() for i in range(4)]
        now = {**cpu, **{n: inp[n].cpu() for n in ADAPTERS}}
        mom = [[to_np(x) for x in opt.moments(i)] for i in range(4)]
        g.replay() if graph else step()
        torch.cuda.synchronize()
        assert ml.moe_get_device_error() == ml.MOE_OK and int(opt.steps) == t
        Y, aux = OL.moe_forward(now, cfg.k, cfg.scale)
        assert rel_err(to_np(buf.Y), Y) <= TOL
        # the router's gradient: through the output's weights and from the balance loss
        x = cpu["logits"].double().numpy()
        loss, counts, n = O.balance_loss(x, aux["ids"], 2, [0, 120, 190])
        assert rel_err(to_np(bal.loss), loss) <= 1e-5 and np.array_equal(bal.counts.cpu().numpy(), counts)
        through, _ = OL.router_backward(cpu["dY"], aux["yp"], aux["ids"], aux["w"], aux["pair_pos"], cfg.E)
        ref = through + O.balance_backward(x, counts, n, np.full(2, 0.25), cfg.k, [0, 120, 190])
        assert rel_err(to_np(bal.dlogits), ref) <= TOL
        # the step with the gradients the layer wrote
        for i, name in enumerate(ADAPTERS):
            w, _, _ = O.adamw(master[i], to_np(opt.grads[i]), mom[i][0], mom[i][1], t, 1e-3, 0.9, 0.999, 1e-8, 0.01)
            got = to_np(opt._part(opt.master, i))
            # 64 u of the update if m's summands did not cancel, 6 u of the weight (test_adamw_gpu.py)
            upd = O.adamw(0.0, np.abs(to_np(opt.grads[i])), np.abs(mom[i][0]), mom[i][1], t, 1e-3, 0.9, 0.999, 1e-8, 0.0)[0]
            past = np.abs(got - w) - 2.0 ** -24 * (64 * np.abs(upd) + 6 * np.abs(w)) - 1e-12
            assert past.max() <= 0
            assert torch.equal(inp[name], opt._part(opt.master, i).to(torch.bfloat16))
            assert not np.array_equal(w, master[i])


def test_gradients_of_adapters_of_an_idle_expert_decay_only():
    cfg = small_config(T=64, m=64, n=32, E=4, k=1, r=8, alpha=8)
    inp, _ = inputs_on(cfg)
    inp["logits"][:, 2] = -100.0                       # expert 2 gets nothing
    buf = ml.alloc_buffers(cfg.T, cfg.m, cfg.n, cfg.E, cfg.k, cfg.r, cfg.scale)
    opt = ml.AdamW([inp[n] for n in ADAPTERS], [buf.dA_gu, buf.dB_gu, buf.dA_d, buf.dB_d], lr=0.1, weight_decay=0.5,
                   master_weights=True)
    before = [opt._part(opt.master, i)[2].clone() for i in range(4)]
    ml.layer_train_step(inp, cfg.k, cfg.scale, buf, opt)
    for i, b in enumerate(before):
        assert torch.allclose(opt._part(opt.master, i)[2], b * 0.95, rtol=1e-6, atol=0)


def test_trained_adapters_served_in_one_batch():
    """Two tenants train the gate/up adapter of a shared expert; both are then served in one batch
    of prompts and single tokens beside the frozen projection."""
    cfg = small_config(T=160, m=128, n=64, E=1, k=1, r=16, alpha=16)
    trained = []
    for seed in (1, 2):
        inp, _ = inputs_on(cfg, seed=seed)
        inp.update({k: v.cuda() for k, v in generate(cfg, seed=0).items() if k in ("W_gu", "W_d")})
        buf = ml.alloc_buffers(cfg.T, cfg.m, cfg.n, 1, 1, cfg.r, cfg.scale)
        opt = ml.AdamW([inp[n] for n in ADAPTERS], [buf.dA_gu, buf.dB_gu, buf.dA_d, buf.dB_d], lr=1e-2, state_bits=8)
        for _ in range(3):
            ml.layer_train_step(inp, 1, cfg.scale, buf, opt)
        trained.append(inp)
    A = torch.cat([t["A_gu"] for t in trained])
    B = torch.cat([t["B_gu"] for t in trained])
    W = trained[0]["W_gu"][0]
    scale = torch.full((2,), cfg.scale, device="cuda")
    X = torch.randn(100, cfg.m, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    off, ad = [0, 60, 61, 62, 95], [1, 0, -1, 0]
    Y = X @ W
    base = to_np(Y)
    ml.moe_lora_requests(X, torch.tensor(ad, dtype=torch.int32, device="cuda"), A, B, scale, Y,
                         torch.tensor(off, dtype=torch.int32, device="cuda"))
    ref = O.lora_requests(to_np(X), ad, to_np(A), to_np(B), to_np(scale), base, off)
    assert rel_err(to_np(Y), ref) <= 2.0 ** -8
    # each tenant's own tokens as the layer itself computes them: GU = X W_gu + c (X A) B
    for tenant, lo, hi in ((1, 0, 60), (0, 62, 95)):
        t = trained[tenant]
        n = hi - lo
        buf = ml.alloc_buffers(n, cfg.m, cfg.n, 1, 1, cfg.r, cfg.scale)
        ml.layer_forward({**t, "X": X[lo:hi].contiguous(), "logits": torch.zeros(n, 1, device="cuda")}, 1, cfg.scale, buf)
        assert rel_err(to_np(buf.save_GU), to_np(Y[lo:hi])) <= TOL


def test_a_step_with_other_gradient_buffers_is_refused():
    cfg = small_config(T=64, m=64, n=32, E=4, k=2, r=8, alpha=8)
    inp, _ = inputs_on(cfg)
    buf, other = (ml.alloc_buffers(cfg.T, cfg.m, cfg.n, cfg.E, cfg.k, cfg.r, cfg.scale) for _ in range(2))
    grads = lambda b: [b.dA_gu, b.dB_gu, b.dA_d, b.dB_d]      # noqa: E731
    params = [inp[n] for n in ADAPTERS]
    for bad in (ml.AdamW(params, grads(other)), ml.AdamW(params, grads(buf)[:3] + grads(other)[3:]),
                ml.AdamW(params[::-1], [torch.zeros_like(p) for p in params[::-1]]),
                ml.AdamW([p.clone() for p in params], grads(buf))):
        before = [p.clone() for p in params]
        with pytest.raises(ValueError):
            ml.layer_train_step(inp, cfg.k, cfg.scale, buf, bad)
        assert int(bad.steps) == 0 and all(torch.equal(a, b) for a, b in zip(before, params))
    # some of the adapters, in any order, beside another layer's
    more = torch.zeros(50, device="cuda")
    opt = ml.AdamW([more, inp["B_d"], inp["A_gu"]], [torch.zeros_like(more), buf.dB_d, buf.dA_gu])
    ml.layer_train_step(inp, cfg.k, cfg.scale, buf, opt)
    assert int(opt.steps) == 1
    # views of separate gate and up adapters
    ad = ml.SplitGateUpAdapters(cfg.E, cfg.m, cfg.n, cfg.r)
    for t in (ad.A_g, ad.B_g, ad.A_u, ad.B_u, ad.A_d, ad.B_d):
        t.normal_(std=0.1)
    split = ad.layer_inputs(inp)
    wide = ml.alloc_buffers(cfg.T, cfg.m, cfg.n, cfg.E, cfg.k, 2 * cfg.r, cfg.scale)
    g = ad.grads(wide)
    opt = ml.AdamW([ad.A_u, ad.B_u, ad.A_d], [g["dA_u"], g["dB_u"], g["dA_d"]])
    start = ad.A_u.clone(), ad.A_g.clone()
    ml.layer_train_step(split, cfg.k, cfg.scale, wide, opt)
    assert not torch.equal(ad.A_u, start[0]) and torch.equal(ad.A_g, start[1])
    opt = ml.AdamW([ad.A_u, ad.A_g], [g["dA_g"], g["dA_u"]])
    with pytest.raises(ValueError):
        ml.layer_train_step(split, cfg.k, cfg.scale, wide, opt)
