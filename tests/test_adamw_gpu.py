"""The AdamW step against the fp64 definition.

Bounds (u = 2^-24): m and v are two products and a sum, 4 u of the summands' absolute values
(6 u for v, whose gradient is squared); the update is a handful of fp32 operations and two
expm1 (a few u each) on m, 64 u of what it would be if m's summands did not cancel; w adds 6 u
of itself.  A bf16 weight adds half a bf16
step, 2^-8 of its value.

8 bits: x (m or sqrt(v)) is off by e <= 4 u (|b1 m0| + |(1 - b1) g|) (m's summands may cancel,
so this is no share of m), or by 6 u of itself for the root.  A block's scale max|x| / 448 is
then off by at most (the block's largest e) / 448 + 4 u of itself, and y = |x| 448 / max by
y (e / |x| + (largest e) / max + 8 u).  A code is the definition's except where the way from the
code below y to the next, plus the random fraction, is that near to one, in widths of a code
(2^-18 more for the subnormal codes, which lose the 20th bit behind them).
"""
import numpy as np
import pytest
import torch

import mixture_experts_lora_b200 as ml
import oracle.train_serve_oracle as O

from gpu_common import ensure_built

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
H = dict(lr=1e-2, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def f64(t):
    return t.detach().double().cpu().numpy().ravel()


class Mirror:
    """The optimizer's state in fp64, taken over before each step and compared after it."""

    def __init__(self, opt):
        self.opt = opt

    def take(self):
        o = self.opt
        self.t = int(o.steps) + 1
        self.before = []
        for i, (p, g) in enumerate(zip(o.params, o.grads)):
            m, v = o.moments(i)
            w = p if o.master is None or p.dtype != BF else o._part(o.master, i)
            self.before.append((f64(w), f64(g), f64(m), f64(v)))

    def check(self, scale=1.0, lr=None, hyper=H):
        o = self.opt
        lr = hyper["lr"] if lr is None else lr
        b1, b2 = hyper["betas"]
        assert int(o.steps) == self.t and int(o._count[1]) == 0
        for i, (w0, g, m0, v0) in enumerate(self.before):
            if len(w0) == 0:
                continue
            g = g * scale
            w, m, v = O.adamw(w0, g, m0, v0, self.t, lr, b1, b2, hyper["eps"], hyper["weight_decay"])
            # m's error is a share of its summands, which may cancel in m itself
            upd = np.abs(O.adamw(0.0, np.abs(g), np.abs(m0), v0, self.t, lr, b1, b2, hyper["eps"], 0.0)[0])
            tol = 64 * U * upd + 6 * U * np.abs(w0)
            p = o.params[i]
            if o.master is not None and p.dtype == BF:
                got = o._part(o.master, i)
                assert np.all(np.abs(f64(got) - w) <= tol)
                assert torch.equal(p, got.to(BF))
            else:
                half = 2.0 ** -8 if p.dtype == BF else U
                assert np.all(np.abs(f64(p) - w) <= tol + half * (np.abs(w) + tol))
            if o.state_bits == 32:
                gm, gv = o.moments(i)
                assert np.all(np.abs(f64(gm) - m) <= 4 * U * (np.abs(b1 * m0) + np.abs((1 - b1) * g)) + 1e-44)
                assert np.all(np.abs(f64(gv) - v) <= 6 * U * v + 1e-44)
                continue
            n, a = len(w0), o.starts[i]
            at = slice(a, a + -(-n // 256) * 256)
            blocks = slice(a // 256, at.stop // 256)
            em = 4 * U * (np.abs(b1 * m0) + np.abs((1 - b1) * g))
            for x, e, codes, scales, u, root in (
                    (m, em, o.exp_avg, o.exp_avg_scale, O.noise(self.t, n)[0], False),
                    (np.sqrt(v), 6 * U * np.sqrt(v), o.exp_avg_sq, o.exp_avg_sq_scale, O.noise(self.t, n)[1], True)):
                got = codes[at].view(torch.uint8).cpu().numpy().astype(np.int64)
                ref, rs, place = O.encode(x, u, root)
                e = np.pad(e, (0, len(got) - n))
                top_e = e.reshape(-1, 256).max(axis=1)
                assert np.all(np.abs(f64(scales[blocks]) - rs) <= top_e / 448 + 4 * U * rs)
                off = got != ref
                top, top_e = np.repeat(np.maximum(rs * 448, 1e-300), 256), np.repeat(top_e, 256)
                y = np.minimum(np.abs(np.pad(x, (0, len(got) - n))) * 448 / top, 448)
                gap = np.maximum(2.0 ** -9, 2.0 ** np.floor(np.log2(np.maximum(y, 2.0 ** -6))) / 8)
                far = (e * 448 / top + y * (top_e / top + 8 * U)) / gap + 2.0 ** -18
                near = np.abs(place - np.round(place)) <= far
                assert not np.any(off & ~near)
                # a code that went the other way is the neighbour (or zero with and without a sign)
                assert np.all(np.abs((got & 0x7F) - (ref & 0x7F))[off] <= 1)


def steps(opt, n=2, seed=1, std=1e-2, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mir = Mirror(opt)
    for _ in range(n):
        for t in opt.grads:
            t.copy_(torch.randn(t.shape, generator=g, device="cuda") * std)
        mir.take()
        opt.step(**kw)
        torch.cuda.synchronize()
        assert ml.moe_get_device_error() == ml.MOE_OK
        mir.check()


def make(shapes, p=BF, g=BF, seed=0, **kw):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    params = [(torch.randn(s, generator=gen, device="cuda") * 0.1).to(p) for s in shapes]
    return ml.AdamW(params, [torch.zeros(s, dtype=g, device="cuda") for s in shapes], **H, **kw)


SHAPES = [(1,), (7,), (8,), (255,), (256,), (257,), (2048,), (2049,), (3, 5, 11), (4, 64, 16), (0,), (6000,)]


@pytest.mark.parametrize("p,g,master", [(BF, BF, False), (BF, BF, True), (BF, F32, True), (BF, F32, False),
                                        (F32, F32, False), (F32, BF, False)])
@pytest.mark.parametrize("bits", [32, 8])
def test_types_and_sizes(p, g, master, bits):
    steps(make(SHAPES, p, g, state_bits=bits, master_weights=master), n=3)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [0, 1, 4, 8])
def test_tensors_packed_back_to_back(bits, offset):
    sizes = [1, 300, 17, 4096, 3, 2050]
    flat = torch.randn(offset + sum(sizes), device="cuda").to(BF)
    gflat = torch.zeros(offset + sum(sizes), device="cuda", dtype=BF)
    cut = np.cumsum([offset] + sizes)
    opt = ml.AdamW([flat[a:b] for a, b in zip(cut, cut[1:])], [gflat[a:b] for a, b in zip(cut, cut[1:])],
                   state_bits=bits, **H)
    head = flat[:offset].clone()
    steps(opt)
    assert torch.equal(flat[:offset], head)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("E,m,n,r", [(3, 48, 32, 8), (2, 80, 48, 16), (5, 33, 7, 5)])
def test_strided_views(bits, E, m, n, r):
    """SplitGateUpAdapters' views: the packed tensors' other blocks stay zero."""
    if r % 8 == 0:
        ad = ml.SplitGateUpAdapters(E, m, n, r)
        A, B = ad.A_gu, ad.B_gu
        params = [ad.A_g, ad.B_g, ad.A_u, ad.B_u, ad.A_d, ad.B_d]
    else:
        A, B = torch.zeros(E, m, 2 * r, dtype=BF, device="cuda"), torch.zeros(E, 2 * r, 2 * n, dtype=BF, device="cuda")
        params = [A[:, :, :r], B[:, :r, :n], A[:, :, r:], B[:, r:, n:]]
    for t in params:
        t.copy_(torch.randn(t.shape, device="cuda") * 0.1)
    gA, gB = torch.randn_like(A), torch.randn_like(B)
    grads = [gA[:, :, :r], gB[:, :r, :n], gA[:, :, r:], gB[:, r:, n:]]
    grads += [torch.randn(t.shape, device="cuda").to(BF) for t in params[4:]]
    steps(ml.AdamW(params, grads, state_bits=bits, **H))
    assert not B[:, :r, n:].any() and not B[:, r:, :n].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_orders_and_broadcast_gradients(bits):
    p = torch.randn(6, 40, 24, device="cuda")
    g = torch.randn(24, 40, 6, device="cuda")
    col = torch.randn(40, 1, device="cuda")
    opt = ml.AdamW([p.transpose(0, 2), torch.randn(40, 50, device="cuda"), torch.randn(64, 33, device="cuda")[:, ::2]],
                   [g, col.expand(40, 50), torch.randn(17, 64, device="cuda").t()], state_bits=bits, **H)
    mir = Mirror(opt)
    mir.take()
    opt.step()
    mir.check()


def test_more_tensors_than_one_launch_holds():
    shapes = [(1 + 37 * i % 700,) for i in range(600)]
    steps(make(shapes, state_bits=32))
    opt = make(shapes[:40], state_bits=8)
    assert len(opt.starts) == 40
    steps(opt)


def test_mixed_types_make_one_step():
    gen = torch.Generator(device="cuda").manual_seed(3)
    params = [torch.randn(300, generator=gen, device="cuda").to(t) for t in (BF, F32, BF, F32)]
    grads = [torch.zeros(300, device="cuda", dtype=t) for t in (BF, F32, F32, BF)]
    opt = ml.AdamW(params, grads, master_weights=True, **H)
    steps(opt, n=3)
    assert int(opt.steps) == 3


def test_grad_scale_lr_tensor_and_first_steps():
    opt = make([(500,), (33, 9)], F32, F32)
    opt.lr = torch.tensor([0.003], device="cuda")
    scale = torch.tensor(0.25, device="cuda")
    mir = Mirror(opt)
    for i in range(3):
        for g in opt.grads:
            g.copy_(torch.randn(g.shape, device="cuda"))
        opt.lr.fill_(0.003 * (i + 1))
        mir.take()
        opt.step(grad_scale=scale)
        mir.check(0.25, float(opt.lr.double()))
    opt.lr = 0.5
    mir.take()
    opt.step()
    mir.check(lr=0.5)
    for bad in (torch.zeros(2, device="cuda"), torch.zeros(1), torch.zeros(1, device="cuda", dtype=BF)):
        with pytest.raises(ValueError):
            opt.step(grad_scale=bad)


@pytest.mark.parametrize("t", [0, 1, 9, 1000, 10 ** 6, 2 ** 33])
@pytest.mark.parametrize("bits", [32, 8])
def test_late_steps_and_other_betas(t, bits):
    hyper = dict(lr=1e-3, betas=(0.0, 0.5), eps=0.0, weight_decay=0.0) if t == 9 else H
    p, g = torch.randn(700, device="cuda"), torch.randn(700, device="cuda")
    opt = ml.AdamW([p], [g], state_bits=bits, **hyper)
    opt.steps.fill_(t)
    mir = Mirror(opt)
    mir.take()
    opt.step()
    mir.check(hyper=hyper)


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_tiny_and_infinite_gradients(bits):
    n = 256 * 6
    p, g = torch.ones(n, device="cuda"), torch.randn(n, device="cuda")
    g[256:512] = 0                        # a block without a gradient
    g[512:768] = 1e-33                    # below what a scale is kept for
    g[768:1024] *= 1e-12
    g[1024] = 1e6                         # one large value beside small ones
    opt = ml.AdamW([p], [g], state_bits=bits, **H)
    mir = Mirror(opt)
    for _ in range(3):
        mir.take()
        opt.step()
        mir.check()
    if bits == 8:
        assert not opt.exp_avg[256:768].view(torch.uint8).any() and not opt.exp_avg_scale[1:3].any()
        # a positive root is never stored as zero
        assert (opt.exp_avg_sq[1025:1280].view(torch.uint8) > 0).all()
    before = p.clone()
    g[1300] = float("inf")
    g[1301] = float("nan")
    opt.step()
    assert torch.isfinite(p[:1280]).all() and not torch.isfinite(p[1301])
    m, v = opt.moments(0)
    hit = ~torch.isfinite(m)
    if bits == 8:                         # the block, and nothing else
        assert hit[1280:].all() and not hit[:1280].any() and not torch.isfinite(v[1280:]).any()
    else:
        assert hit.nonzero().ravel().tolist() == [1300, 1301]
    assert torch.isfinite(before).all()


def test_slow_averages_move_in_8_bits():
    """sqrt(v) of a gradient that stopped falls by 0.05% a step, far less than a code."""
    g = torch.full((256 * 64,), 1e-3, device="cuda")
    g[::256] = 1.0                        # holds the blocks' scales
    opt = ml.AdamW([torch.zeros_like(g)], [g], state_bits=8, lr=0.0)
    opt.exp_avg_sq.view(torch.uint8).fill_(0x60)          # 32 of 448
    opt.exp_avg_sq.view(torch.uint8)[::256] = 0x7E
    opt.exp_avg_sq_scale.fill_(1 / 448)
    opt.steps.fill_(5000)
    g[1:].fill_(0.0)
    g[::256] = 1.0
    for _ in range(1000):
        opt.step()
    _, v = opt.moments(0)
    rest = v.sqrt().view(-1, 256)[:, 1:].mean().item()
    # 16320 elements: the mean of their last roundings (a code is 1/8 of the value) is within 1%
    assert abs(rest / (32 / 448 * 0.999 ** 500) - 1) < 0.03


def test_in_a_graph_and_on_another_stream():
    def fresh():
        o = make([(40, 70), (513,)], state_bits=8, seed=5)
        for i, g in enumerate(o.grads):
            g.copy_(torch.randn(g.shape, generator=torch.Generator().manual_seed(i)))
        return o
    want, got = fresh(), fresh()
    for _ in range(4):
        want.step()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got.step(stream=st)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.step()
    assert int(got.steps) == 1               # capturing is not running
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert int(got.steps) == 4
    for a, b in zip(want.params, got.params):
        assert torch.equal(a, b)
    for k in ("exp_avg", "exp_avg_sq"):
        assert torch.equal(getattr(want, k).view(torch.uint8), getattr(got, k).view(torch.uint8))


@pytest.mark.parametrize("bits,master", [(32, True), (8, False)])
def test_state_dict(bits, master):
    a = make([(100,), (3, 300)], state_bits=bits, master_weights=master)
    steps(a)
    b = make([(100,), (3, 300)], state_bits=bits, master_weights=master, seed=9)
    for x, y in zip(b.params + b.grads, a.params + a.grads):
        x.copy_(y)
    b.load_state_dict(a.state_dict())
    a.step()
    b.step()
    for x, y in zip(b.params, a.params):
        assert torch.equal(x, y)
    assert int(b.steps) == int(a.steps) == 3
    with pytest.raises(ValueError):
        make([(100,)], state_bits=bits, master_weights=master).load_state_dict(a.state_dict())


def test_refusals():
    p = torch.zeros(8, 8, device="cuda", dtype=BF)
    for params, grads in (([p], [p[:4]]), ([p.half()], [p]), ([p], [p.double()]), ([p, p], [p, p]),
                          ([p[:1].expand(8, 8)], [p]), ([p], [p.cpu()]), ([p], []),
                          ([p.view(-1).as_strided((8, 8), (4, 1))], [p]), ([p.view(-1).unfold(0, 16, 8)], [torch.zeros(7, 16).to(p)])):
        with pytest.raises(ValueError):
            ml.AdamW(params, grads)
    with pytest.raises(ml.MoEError):
        ml.AdamW([p], [p], betas=(1.0, 0.9)).step()


def test_trains_a_small_problem():
    """Runs: the weights follow torch's own AdamW on the same gradients (fp32, 20 steps)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    p = torch.randn(64, 32, generator=g, device="cuda")
    q = torch.nn.Parameter(p.double())
    ref = torch.optim.AdamW([q], lr=1e-2, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
    opt = ml.AdamW([p], [torch.zeros_like(p)], **H)
    for _ in range(20):
        grad = torch.randn(64, 32, generator=g, device="cuda")
        opt.grads[0].copy_(grad)
        q.grad = grad.double()
        opt.step()
        ref.step()
    # 20 steps, each 70 u of an update below 0.1 and of weights below 8
    assert (p.double() - q.detach()).abs().max() <= 20 * 70 * U * 8


@pytest.mark.parametrize("bits", [8, 32])
def test_elements_past_32_bits(bits):
    """A tensor of more than 2^31 elements whose last ones move as they do in a tensor of their own."""
    n, tail = (1 << 31) + 1000, 700
    p, g = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(4)
    sp = torch.randn(tail, generator=gen).bfloat16().cuda()
    sg = torch.randn(tail, generator=gen).bfloat16().cuda()
    p[-tail:], g[-tail:] = sp, sg
    kw = dict(lr=0.01, weight_decay=0.1, state_bits=bits)
    ml.AdamW([p], [g], **kw).step()
    ml.AdamW([sp], [sg], **kw).step()
    torch.cuda.synchronize()
    assert torch.equal(p[-tail:], sp)
    assert not p[:-tail].any()


@pytest.mark.parametrize("e", [-126, -125, -120, -110, -103, -101, -100, -99, -80, -1, 0])
def test_the_root_of_small_moments(e):
    """Groups of eight and single elements take the same root: with w = 0 and eps = 0 the weight shows it
    to the last bits.  v from 2^e up to twice that; both forms round every operation alike."""
    n = 4096
    g = torch.Generator(device="cuda").manual_seed(e + 200)
    v = torch.ldexp(torch.rand(n, generator=g, device="cuda") + 1.0, torch.tensor(e + 1.0, device="cuda"))
    m = torch.sqrt(v) * (torch.rand(n, generator=g, device="cuda") + 0.5)
    out = []
    for offset in (0, 1):                    # aligned: groups of eight; one off: single elements
        p = torch.zeros(n + offset, device="cuda")[offset:]
        opt = ml.AdamW([p], [torch.zeros(n + offset, device="cuda")[offset:]], lr=1.0, betas=(0.5, 0.5), eps=0.0,
                       weight_decay=0.0)
        opt.exp_avg.copy_(m)
        opt.exp_avg_sq.copy_(v)
        opt.step()
        assert torch.equal(opt.exp_avg_sq, v / 2) and torch.equal(opt.exp_avg, m / 2)
        out.append(p)
    assert torch.equal(out[0], out[1])


def test_the_root_of_every_moment_of_two_octaves():
    """All 2^24 floats of [1, 4) as v, groups of eight against single elements."""
    n = 1 << 24
    v = (torch.arange(n, dtype=torch.int32, device="cuda") + 0x3F800000).view(torch.float32)
    assert v[0] == 1 and v[-1] < 4 and v[-1] > 3.9999995
    out = []
    for offset in (0, 1):
        p = torch.zeros(n + offset, device="cuda")[offset:]
        opt = ml.AdamW([p], [torch.zeros(n + offset, device="cuda")[offset:]], lr=1.0, betas=(0.5, 0.5), eps=0.0,
                       weight_decay=0.0)
        opt.exp_avg.copy_(v.flip(0))
        opt.exp_avg_sq.copy_(v * 2)
        opt.step()
        assert torch.equal(opt.exp_avg_sq, v)
        out.append(p)
    assert torch.equal(out[0], out[1])


@pytest.mark.parametrize("which", ["params", "grads"])
def test_tensors_that_were_given_other_memory(which):
    opt = make([(40,), (3, 70), (513,)], F32, F32)
    for g in opt.grads:
        g.fill_(1.0)
    opt.step()
    t = getattr(opt, which)[1]
    old = t.detach()
    before = [p.clone() for p in opt.params]
    t.data = t.detach().clone()
    for call in (opt.step, lambda: opt.load_state_dict(opt.state_dict())):
        with pytest.raises(ValueError):
            call()
    assert int(opt.steps) == 1 and all(torch.equal(p, b) for p, b in zip(opt.params, before))
    t.data = old
    opt.step()
    assert int(opt.steps) == 2 and not torch.equal(opt.params[1], before[1])


def test_other_memory_is_seen_among_many_tensors():
    """Where a step does not look at all tensors, the next ones do; meanwhile the old memory is kept."""
    opt = make([(10 + i,) for i in range(100)], F32, F32)
    at = opt.params[70].data_ptr()
    opt.params[70].data = opt.params[70].clone()
    junk = [torch.zeros(80, device="cuda") for _ in range(50)]
    assert all(j.data_ptr() != at for j in junk)
    with pytest.raises(ValueError):
        for _ in range(-(-200 // ml.LOOKED_AT)):
            opt.step()
    torch.cuda.synchronize()
    assert not any(j.any() for j in junk)


def test_parameters_that_share_memory_are_refused():
    flat = torch.zeros(400, device="cuda")
    grid = torch.zeros(6, 20, 32, device="cuda", dtype=BF)
    def make_over(*params):
        return ml.AdamW(list(params), [torch.zeros(p.shape, dtype=p.dtype, device="cuda") for p in params], **H)
    for bad in ((flat[0:10], flat[5:15]), (flat[5:15], flat[0:300], flat[390:]), (flat[:10], flat[9:10]),
                (grid[:, :, :16], grid[:, :, 15:]), (grid[:, :8], grid), (grid[:, ::2, :8], grid[:, 1:19, 4:20]),
                (flat[::2], flat[2:3]), (flat[:100].view(torch.bfloat16), flat[99:120]),
                (flat[::4], flat[1::4], flat[2::4], flat[6::4])):
        with pytest.raises(ValueError):
            make_over(*bad)
    for good in ((flat[0:10], flat[10:15]), (grid[:, :, :16], grid[:, :, 16:]), (grid[:, ::2, :16], grid[:, 1::2], grid[:, ::2, 16:]),
                 (flat[::2], flat[1::2]), (flat[:100].view(torch.bfloat16), flat[100:120]), (flat[5:5], flat[0:10], flat[5:5]),
                 (flat[::4], flat[1::4], flat[2::4], flat[3::4])):
        steps(make_over(*good), n=1)


@pytest.mark.parametrize("bits", [32, 8])
def test_master_weights_follow_weights_that_are_loaded(bits):
    opt = make([(300,), (8, 40)], state_bits=bits, master_weights=True)
    steps(opt, n=1)
    for p in opt.params:
        p.fill_(3.0)
    opt.refresh_master()
    for i in range(2):
        assert (opt._part(opt.master, i) == 3.0).all()
    steps(opt, n=1)                          # (checked against a step from these weights)
    for p in opt.params:
        assert ((p.float() - 3.0).abs() < 0.1).all()
    mixed = ml.AdamW([torch.ones(9, device="cuda"), torch.ones(9, device="cuda", dtype=BF)],
                     [torch.ones(9, device="cuda"), torch.ones(9, device="cuda", dtype=BF)], master_weights=True)
    mixed.params[1].fill_(2.0)
    mixed.refresh_master()
    assert (mixed._part(mixed.master, 1) == 2.0).all() and not mixed._part(mixed.master, 0).any()
    none = make([(5,)], F32, F32)
    none.refresh_master()                    # nothing to refresh
    assert none.master is None


@pytest.mark.parametrize("sizes,master", [((2200001,), False), ((1500000, 256, 1400300), True), ((11_000_255,), True)])
def test_8_bit_states_of_large_tensors(sizes, master):
    """Tensors of which a warp walks several blocks in a row, with a part of a block at the end: codes
    and scales of two steps from moments that are not zero."""
    opt = make([(n,) for n in sizes], state_bits=8, master_weights=master)
    opt.steps.fill_(50)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for i, (a, n) in enumerate(zip(opt.starts, sizes)):       # (the elements behind a tensor's end stay zero)
        for codes, top in ((opt.exp_avg, 256), (opt.exp_avg_sq, 128)):
            draw = torch.randint(0, top, (n,), generator=gen, device="cuda", dtype=torch.int32)
            codes[a:a + n].view(torch.uint8).copy_(torch.where(draw & 0x7F == 0x7F, draw - 1, draw))
    opt.exp_avg_scale.copy_(torch.rand(opt.exp_avg_scale.shape, generator=gen, device="cuda") * 1e-4 + 1e-6)
    opt.exp_avg_sq_scale.copy_(torch.rand(opt.exp_avg_sq_scale.shape, generator=gen, device="cuda") * 1e-4 + 1e-6)
    steps(opt, n=2)


@pytest.mark.parametrize("p,master", [(BF, True), (F32, False)])
def test_more_elements_than_resident_blocks_take_at_once(p, master):
    """Over 64 chunks of 2048 elements per SM: the 32-bit step's blocks go on to others."""
    steps(make([(20_000_003,), (300,)], p, F32, master_weights=master), n=2)


@pytest.mark.parametrize("bits", [32, 8])
def test_the_smallest_eps(bits):
    """Elements that never had a gradient stay where they are (0 / eps = 0), whatever eps."""
    p = torch.randn(600, device="cuda")
    g = torch.zeros(600, device="cuda")
    g[300] = 1e-3
    before = p.clone()
    opt = ml.AdamW([p], [g], lr=0.1, eps=2.0 ** -126, weight_decay=0.0, state_bits=bits)
    opt.step()
    moved = (p != before).nonzero().ravel().tolist()
    assert moved == [300] and torch.isfinite(p).all()
    with pytest.raises(ml.MoEError):
        ml.AdamW([p], [g], eps=2.0 ** -127, state_bits=bits).step()


@pytest.mark.parametrize("g", [BF, F32])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [0, 1])
def test_moments_are_rounded_operation_by_operation(bits, offset, g):
    """Bit for bit what separate fp32 operations give, in groups of eight and element by element."""
    n = 256 * 1500 + 40
    gen = torch.Generator(device="cuda").manual_seed(3)
    grad = (torch.randn(n + offset, generator=gen, device="cuda") * 1e-3).to(g)[offset:]
    opt = ml.AdamW([torch.zeros(n + offset, device="cuda")[offset:]], [grad], state_bits=bits, **H)
    if bits == 32:
        opt.exp_avg[:n] = torch.randn(n, generator=gen, device="cuda") * 1e-4
        opt.exp_avg_sq[:n] = (torch.randn(n, generator=gen, device="cuda") * 1e-3).square()
    else:
        for codes, top in ((opt.exp_avg, 256), (opt.exp_avg_sq, 128)):
            draw = torch.randint(0, top, (n,), generator=gen, device="cuda", dtype=torch.int32)
            codes[:n].view(torch.uint8).copy_(torch.where(draw & 0x7F == 0x7F, draw - 1, draw))
        opt.exp_avg_scale.copy_(torch.rand(1501, generator=gen, device="cuda") * 1e-6)
        opt.exp_avg_sq_scale.copy_(torch.rand(1501, generator=gen, device="cuda") * 1e-5)
    m, v = (x.clone() for x in opt.moments(0))
    f = lambda x: torch.tensor(x, dtype=F32, device="cuda")      # noqa: E731
    b1, b2 = H["betas"]
    x = grad.float()
    m = torch.add(torch.mul(m, f(b1)), torch.mul(x, f(1 - b1)))
    v = torch.add(torch.mul(v, f(b2)), torch.mul(torch.mul(x, x), f(1 - b2)))
    opt.step()
    if bits == 32:
        assert torch.equal(opt.exp_avg[:n], m) and torch.equal(opt.exp_avg_sq[:n], v)
        return
    inv = f(1.0) / f(448.0)
    for y, scale in ((m.abs(), opt.exp_avg_scale), (v.sqrt(), opt.exp_avg_sq_scale)):
        top = torch.nn.functional.pad(y, (0, -n % 256)).view(-1, 256).amax(1)
        assert torch.equal(scale, top * inv)
