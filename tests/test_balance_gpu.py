"""The router's balance loss and its gradient against the fp64 definition.

Bounds (u = 2^-24, fp32 rounding): a probability is an exponential over a sum of E positive
terms, relative error (E + 16) u; the loss is a sum of at most T k such positive products, each
addition adding at most u, so (E + T + 64) u of its value bounds it.  A gradient entry
p (f - sum_j p_j f_j) is at most (3 E + 64) u p (f + sum_j p_j f_j) off, f >= 0 up to the sign of
the upstream gradient.
"""
import numpy as np
import pytest
import torch

import mixture_experts_lora_b200 as ml
import oracle.train_serve_oracle as O
from moe_inputs import CONFIGS

from gpu_common import ensure_built, inputs_on, run_layer

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


class Case:
    def __init__(self, T, E, k, off=None, mask=None, seed=0, ids=None, logits=None, spread=1.0, lead=0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.E, self.k = T, E, k
        self.logits = torch.randn(T, E, generator=g) * spread if logits is None else logits
        order = torch.randn(T, E, generator=g).argsort(dim=1)[:, :k]
        self.ids = (order if ids is None else ids).to(torch.int32)
        self.off = off
        self.S = 1 if off is None else len(off) - 1
        self.mask = mask
        self.dloss = torch.randn(self.S, generator=g)
        self.lead = lead            # elements in front of the logits (alignment)

    def on_gpu(self, t):
        if t is None:
            return None
        if self.lead and t.dim() == 2 and t.dtype == torch.float32:
            flat = torch.empty(t.numel() + self.lead, device="cuda")
            v = flat[self.lead:].view(t.shape)
            v.copy_(t)
            return v
        return t.cuda()

    def run(self, accumulate=None, stream=None):
        S, E = self.S, self.E
        x, ids, mask = self.on_gpu(self.logits), self.ids.cuda(), self.on_gpu(self.mask)
        off = None if self.off is None else torch.tensor(self.off, dtype=torch.int32, device="cuda")
        loss = torch.full((S,), float("nan"), device="cuda")
        counts = torch.full((S, E), -1, dtype=torch.int32, device="cuda")
        n = torch.full((S,), -1, dtype=torch.int32, device="cuda")
        ws = torch.full((ml.moe_balance_workspace_bytes(self.T, E, S),), 0xFF, dtype=torch.uint8, device="cuda")
        grad = self.on_gpu(torch.full((self.T, E), float("nan")) if accumulate is None else accumulate)
        ml.moe_balance_loss(x, ids, loss, counts, n, ws, off, mask, stream)
        ml.moe_balance_loss_backward(x, counts, n, self.dloss.cuda(), self.k, grad, off, mask,
                                     accumulate is not None, stream)
        torch.cuda.synchronize()
        assert ml.moe_get_device_error() == ml.MOE_OK
        return loss.cpu(), counts.cpu(), n.cpu(), grad.cpu()

    def check(self, got, base=None):
        loss, counts, n, grad = (t.double().numpy() for t in got)
        x, ids = self.logits.double().numpy(), self.ids.numpy()
        mask = None if self.mask is None else self.mask.numpy()
        rl, rc, rn = O.balance_loss(x, ids, self.S, self.off, mask)
        assert np.array_equal(counts, rc) and np.array_equal(n, rn)
        assert np.all(np.abs(loss - rl) <= (self.E + self.T + 64) * U * rl)
        d = self.dloss.double().numpy()
        rg = O.balance_backward(x, rc, rn, d, self.k, self.off, mask)
        # p (f + sum p f): the same expression with a plus, from the definition's parts
        p = O.softmax(x)
        bound = np.zeros_like(rg)
        for s in range(self.S):
            rows = O._rows(self.T, self.off, mask, s)
            if len(rows):
                f = rc[s] * (abs(d[s]) * self.E / (self.k * len(rows) ** 2))
                bound[rows] = p[rows] * (f + p[rows] @ f[:, None])
        tol = (3 * self.E + 64) * U * bound
        if base is not None:
            rg = rg + base.double().numpy()
            tol = tol + U * np.abs(rg)
        assert np.all(np.abs(grad - rg) <= tol)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 3, 3), (31, 32, 4), (257, 7, 1), (64, 33, 5), (100, 64, 8),
                                   (70, 127, 8), (513, 128, 8), (40, 130, 32), (129, 256, 8), (33, 257, 3), (20, 512, 6),
                                   (17, 1000, 32), (9, 1024, 2), (1000, 20, 4), (300, 12, 2), (65, 36, 8)])
def test_one_sequence(T, E, k):
    c = Case(T, E, k)
    c.check(c.run())


@pytest.mark.parametrize("off", [[0, 50], [0, 0, 100], [0, 1, 2, 3, 40, 40, 40, 99], [5, 5, 60, 96],
                                 list(range(101)), [0] * 70 + [31, 32, 33, 64, 100]])
@pytest.mark.parametrize("E", [24, 129])
def test_packed_sequences(off, E):
    c = Case(100, E, 4, off=off, seed=len(off))
    got = c.run()
    c.check(got)
    assert not got[3][:off[0]].any() and not got[3][off[-1]:].any()


def test_many_sequences_over_many_windows():
    g = np.random.default_rng(5)
    cut = np.sort(g.integers(0, 20001, size=700)).tolist()
    c = Case(20000, 40, 3, off=[0] + cut + [20000], mask=torch.from_numpy(g.random(20000) > 0.2), seed=6)
    c.check(c.run())


@pytest.mark.parametrize("T,S,E", [(50, 200000, 16), (900, 5000, 40), (1024, 4, 32), (1025, 4, 32), (2049, 3, 8)])
def test_many_empty_sequences(T, S, E):
    """Runs of empty sequences inside a window; batches at the border of one window."""
    g = np.random.default_rng(S)
    # ends at a few places only: long runs of sequences that begin and end at one row
    cut = np.sort(g.choice(g.integers(0, T + 1, size=7), size=S - 1)).tolist()
    c = Case(T, E, 3, off=[0] + cut + [T], seed=T)
    c.check(c.run())


@pytest.mark.parametrize("E", [8, 48, 300])
def test_masked_rows_are_not_looked_at(E):
    T, off = 90, [0, 30, 60, 80]
    mask = torch.rand(T, generator=torch.Generator().manual_seed(1)) > 0.5
    mask[30:60] = False                               # a sequence without valid rows
    c = Case(T, E, 2, off=off, mask=mask, seed=2)
    want = c.run()
    c.check(want)
    assert want[0][1] == 0 and want[2][1] == 0 and not want[3][30:60].any()
    x, ids = c.logits.clone(), c.ids.clone()
    dead = ~mask
    dead[80:] = True                                  # and rows of no sequence
    x[dead] = torch.tensor([float("nan"), float("inf"), -float("inf")]).repeat(E)[:E]
    ids[mask.logical_not()] = -7
    c.logits, c.ids = x, ids
    for a, b in zip(want, c.run()):
        assert torch.equal(a, b)
    c.mask = c.mask.to(torch.uint8) * 3               # any non-zero byte counts
    assert torch.equal(c.run()[0], want[0])


def test_logits_at_the_ends_of_their_range():
    T, E = 40, 16
    low = torch.finfo(torch.float32).min
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(3))
    x[0], x[1, 1:], x[2, :8], x[3] = low, low, -float("inf"), 3e38
    x[4, :], x[4, 5] = -float("inf"), 1.0
    x[5] = -float("inf")                              # no finite logit: no probability, no gradient
    c = Case(T, E, 2, logits=x)
    got = c.run()
    c.check(got)
    assert not got[3][5].any()
    x[6, 2] = float("nan")                            # shows in the loss and in its own row's gradient
    loss, _, _, grad = c.run()
    assert torch.isnan(loss).all() and torch.isnan(grad[6]).all()
    assert torch.equal(grad[:6], got[3][:6]) and torch.equal(grad[7:], got[3][7:])


def test_the_same_expert_twice_and_collapsed_routing():
    ids = torch.full((50, 4), 5)
    c = Case(50, 9, 4, ids=ids)
    c.check(c.run())


@pytest.mark.parametrize("E,lead", [(16, 0), (16, 1), (128, 3), (50, 2)])
def test_accumulate_and_alignment(E, lead):
    T = 77
    mask = torch.arange(T) % 5 != 0
    c = Case(T, E, 3, off=[0, 20, 70], mask=mask, lead=lead)
    base = torch.randn(T, E, generator=torch.Generator().manual_seed(9))
    got = c.run(accumulate=base)
    c.check(got, base)
    still = ~mask
    still[70:] = True
    assert torch.equal(got[3][still], base[still])    # rows that count for nothing stay as they were
    c.check(c.run())


def test_no_rows():
    c = Case(0, 8, 2)
    loss, counts, n, _ = c.run()
    assert loss.item() == 0 and not counts.any() and n.item() == 0
    c = Case(0, 8, 2, off=[0, 0, 0])
    loss, counts, n, _ = c.run()
    assert not loss.any() and not counts.any() and not n.any()


def test_bad_ids_and_offsets_are_reported():
    ids = torch.zeros(10, 2, dtype=torch.int64)
    ids[4, 1] = 8
    for c in (Case(10, 8, 2, ids=ids), Case(10, 8, 2, off=[0, 6, 4, 10]), Case(10, 8, 2, off=[0, 5, 11]),
              Case(10, 8, 2, off=[-3, 5, 10])):
        with pytest.raises(AssertionError):
            c.run()
        assert ml.moe_get_device_error() == ml.MOE_OK      # cleared by the read
    with pytest.raises(ml.MoEError):
        c = Case(10, 8, 2)
        ml.moe_balance_loss(c.logits.cuda(), c.ids.cuda(), torch.empty(1, device="cuda"),
                            torch.empty(1, 8, dtype=torch.int32, device="cuda"),
                            torch.empty(1, dtype=torch.int32, device="cuda"),
                            torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_repeatable_on_streams_and_in_a_graph():
    c = Case(5000, 128, 8, off=[0, 1000, 1000, 4100, 4990], seed=4)
    want = c.run()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for a, b in zip(want, c.run(stream=st)):
        assert torch.equal(a, b)
    x, ids, d = c.logits.cuda(), c.ids.cuda(), c.dloss.cuda()
    off = torch.tensor(c.off, dtype=torch.int32, device="cuda")
    out = [torch.empty(4, device="cuda"), torch.empty(4, 128, dtype=torch.int32, device="cuda"),
           torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(5000, 128, device="cuda")]
    ws = torch.empty(ml.moe_balance_workspace_bytes(5000, 128, 4), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ml.moe_balance_loss(x, ids, out[0], out[1], out[2], ws, off)
        ml.moe_balance_loss_backward(x, out[1], out[2], d, 8, out[3], off)
    for _ in range(2):
        for t in out:
            t.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b.cpu())
    x.copy_(c.logits.flip(0))                          # a replay reads what is there then
    graph.replay()
    c.logits = c.logits.flip(0)
    for a, b in zip(c.run(), out):
        assert torch.equal(a, b.cpu())


@pytest.mark.parametrize("name", ["tiny", "qwen3_30b_a3b"])
def test_beside_the_router_backward(name):
    """The routing's own ids; the gradient added to moe_router_backward's."""
    cfg = CONFIGS[name]
    inp, cpu = inputs_on(cfg)
    buf = run_layer(inp, cfg)
    bal = ml.alloc_balance(cfg.T, cfg.E, 1, weight=0.01)
    ml.moe_balance_loss(inp["logits"], buf.ids, bal.loss, bal.counts, bal.n_tokens, bal.ws)
    ml.moe_router_backward(inp["dY"], buf.Y_sorted, buf.ids, buf.w, buf.pair_pos, cfg.E, bal.dlogits)
    base = bal.dlogits.clone()
    ml.moe_balance_loss_backward(inp["logits"], bal.counts, bal.n_tokens, bal.dloss, cfg.k, bal.dlogits,
                                 accumulate=True)
    torch.cuda.synchronize()
    assert ml.moe_get_device_error() == ml.MOE_OK
    assert torch.equal(bal.counts[0], buf.counts)      # the permutation's counts
    c = Case(cfg.T, cfg.E, cfg.k, ids=buf.ids.cpu().long(), logits=cpu["logits"])
    c.dloss = bal.dloss.cpu()
    c.check((bal.loss.cpu(), bal.counts.cpu(), bal.n_tokens.cpu(), bal.dlogits.cpu()), base.cpu())


@pytest.mark.parametrize("T,E,k,cuts", [(40000, 256, 8, ()), (40001, 130, 4, (17, 20000)), (20000, 1000, 6, (19999,)),
                                        (30000, 384, 2, ()), (50000, 60, 4, (1, 49000)), (20000, 1023, 3, (5000, 10000)),
                                        (60000, 33, 2, ()), (6000, 128, 8, (3000,))])
def test_few_sequences_over_many_windows(T, E, k, cuts):
    c = Case(T, E, k, None if not cuts else [0, *cuts, T])
    c.check(c.run())


def test_logits_past_32_bits():
    """More than 2^31 logits, the last rows a sequence of their own: the same as those rows alone.
    A row sum runs over at most 1000 rows a warp and 50 partial sums, so 2000 u + E u bounds the rest."""
    T, E, k, tail = (1 << 21) + 3000, 1024, 2, 40
    dev = dict(device="cuda")
    x, grad = torch.zeros(T, E, **dev), torch.empty(T, E, **dev)
    ids = torch.zeros(T, k, dtype=torch.int32, **dev)
    ids[:, 1] = 1
    small = Case(tail, E, k, seed=3)
    x[-tail:], ids[-tail:] = small.logits.cuda(), small.ids.cuda()
    small.dloss = torch.ones(1)
    want = small.run()
    off = torch.tensor([0, T - tail, T], dtype=torch.int32, **dev)
    loss, counts, n = torch.empty(2, **dev), torch.empty(2, E, dtype=torch.int32, **dev), torch.empty(2, dtype=torch.int32, **dev)
    ws = torch.empty(ml.moe_balance_workspace_bytes(T, E, 2), dtype=torch.uint8, **dev)
    ml.moe_balance_loss(x, ids, loss, counts, n, ws, off)
    ml.moe_balance_loss_backward(x, counts, n, torch.ones(2, **dev), k, grad, off)
    assert ml.moe_get_device_error() == ml.MOE_OK
    assert torch.equal(counts[1:].cpu(), want[1]) and n.tolist() == [T - tail, tail]
    assert counts[0, :2].tolist() == [T - tail] * 2 and not counts[0, 2:].any()
    tol = (2000 + E) * U
    assert abs(loss[1].item() - want[0].item()) <= 2 * tol * want[0].item() and abs(loss[0].item() - 1) <= tol
    small.check((want[0], want[1], want[2], grad[-tail:].cpu()))
    # uniform rows: E / (k n^2) (count - n k / E) / E, the counts n, n, 0, 0, ...
    N = T - tail
    for row in (0, N // 2, N - 1):
        r = grad[row].double().cpu()
        f = torch.zeros(E, dtype=torch.float64)
        f[:2] = N
        ref = (f - f.sum() / E) / (k * N * N)
        assert (r - ref).abs().max() <= (3 * E + 64) * U * 2 / (k * N)


@pytest.mark.parametrize("E,long,short", [(64, 18945, 18944), (128, 131072, 130832), (300, 9473, 9472), (40, 600, 33)])
def test_one_workspace_for_batches_of_many_lengths(E, long, short):
    """The workspace of the longest batch serves shorter ones, and no byte behind it is written."""
    need = ml.moe_balance_workspace_bytes(long, E, 3)
    whole = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    for T in (long, short):
        c = Case(T, E, 2, off=[0, T // 3, T // 2, T], seed=E)
        x, ids = c.logits.cuda(), c.ids.cuda()
        off = torch.tensor(c.off, dtype=torch.int32, device="cuda")
        loss, n = torch.empty(3, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
        counts = torch.empty(3, E, dtype=torch.int32, device="cuda")
        ml.moe_balance_loss(x, ids, loss, counts, n, whole[:need], off)
        torch.cuda.synchronize()
        assert ml.moe_get_device_error() == ml.MOE_OK
        rl, rc, rn = O.balance_loss(c.logits.double().numpy(), c.ids.numpy(), 3, c.off, None)
        assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(n.cpu().numpy(), rn)
        assert (whole[need:] == 0x5A).all()


@pytest.mark.parametrize("T,E,k,cuts", [(60000, 33, 2, ()), (131071, 128, 8, ()), (131071, 128, 8, (40000, 40001, 100000)),
                                        (100000, 8, 2, ()), (30000, 384, 2, (29000,)), (16384, 1024, 8, ())])
def test_the_loss_of_long_batches(T, E, k, cuts):
    """Nothing of a long sum is lost.  A probability is (E + 16) u off.  It is added up over the rows of a
    window that its warp takes, 32 lanes and 8 warps, and the windows, of which there are at most 592, or 296
    above 256 experts; then E products.  A lost window would be more than ten times the bound."""
    c = Case(T, E, k, None if not cuts else [0, *cuts, T], seed=T + E)
    loss = c.run()[0].double().numpy()
    ref, _, _ = O.balance_loss(c.logits.double().numpy(), c.ids.numpy(), c.S, c.off, None)
    windows = 592 if E <= 256 else 296
    chain = 2 * E + 16 + T // windows + 1 + 5 + 8 + windows + 16
    assert np.all(np.abs(loss - ref) <= chain * U * ref)
    assert chain * U < 1 / windows / 10


@pytest.mark.parametrize("T,E,k,off", [(64, 2, 1, None), (132, 1024, 15, [0, 50, 51, 90, 132]), (74, 26, 2, [0, 1, 2, 3, 40, 74]),
                                       (300, 16, 8, list(range(0, 301, 3))), (3000, 219, 26, [0, 2000, 3000])])
@pytest.mark.parametrize("accumulate", [False, True])
def test_the_gradient_of_peaked_rows(T, E, k, off, accumulate):
    """Rows that one expert has nearly whole, beside experts that the sequence never used: the gradient of
    those is a small probability times a count, and neither cancels."""
    c = Case(T, E, k, off=off, seed=E, spread=5.0)
    base = torch.randn(T, E, generator=torch.Generator().manual_seed(9)) * 1e-5 if accumulate else None
    c.check(c.run(accumulate=base), base)
