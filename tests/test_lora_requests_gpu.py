"""The adapters of many requests against the fp64 definition.

Bound of an entry: half a bf16 step of the result (2^-8); X A and its product with B in fp32
with chains of at most K / 8 + 300 additions, u = 2^-24 each, of the products' absolute values;
X A as the sum of two bf16, 2^-17 of itself.
"""
import numpy as np
import pytest
import torch

import mixture_experts_lora_b200 as ml
import oracle.train_serve_oracle as O

from gpu_common import ensure_built

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


class Case:
    def __init__(self, T, K, N, r, n, adapters, off=None, seed=0, ldx=0, ldy=0):
        g = torch.Generator().manual_seed(seed)
        self.Xs = torch.randn(T, K + ldx, generator=g).to(BF).cuda()
        self.Ys = torch.randn(T, N + ldy, generator=g).to(BF).cuda()
        self.X, self.Y = self.Xs[:, ldx:], self.Ys[:, ldy:]
        self.A = (torch.randn(n, K, r, generator=g) / K ** 0.5).to(BF).cuda()
        self.B = torch.randn(n, r, N, generator=g).to(BF).cuda()
        self.scale = (torch.rand(n, generator=g) + 0.5).cuda()
        self.adapters, self.off, self.ldy = adapters, off, ldy
        self.ad = torch.tensor(adapters, dtype=torch.int32, device="cuda")
        self.offs = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")

    def call(self, stream=None):
        ml.moe_lora_requests(self.X, self.ad, self.A, self.B, self.scale, self.Y, self.offs, stream)

    def run(self):
        self.before = self.Ys.clone()
        self.call()
        torch.cuda.synchronize()
        assert ml.moe_get_device_error() == ml.MOE_OK
        return self

    def check(self):
        f = lambda t: t.double().cpu().numpy()      # noqa: E731
        X, A, B, c, Y0 = f(self.X), f(self.A), f(self.B), f(self.scale), f(self.before[:, self.ldy:])
        ref = O.lora_requests(X, self.adapters, A, B, c, Y0, self.off)
        zero = np.zeros_like(Y0)
        both = O.lora_requests(np.abs(X), self.adapters, np.abs(A), np.abs(B), c, zero, self.off)
        K = X.shape[1]
        tol = 2.0 ** -8 * np.abs(ref) + ((K / 8 + 300) * U + 2.0 ** -17) * both
        assert np.all(np.abs(f(self.Y) - ref) <= tol)
        # rows without an adapter, rows of no request and the other columns: bit for bit
        idle = torch.ones(X.shape[0], dtype=torch.bool)
        for s, a in enumerate(self.adapters):
            lo, hi = (s, s + 1) if self.off is None else self.off[s:s + 2]
            if a >= 0:
                idle[lo:hi] = False
        bits = lambda t: t.view(torch.int16)        # noqa: E731
        assert torch.equal(bits(self.Ys)[idle.cuda()], bits(self.before)[idle.cuda()])
        assert torch.equal(bits(self.Ys[:, :self.ldy]), bits(self.before[:, :self.ldy]))


@pytest.mark.parametrize("K,N,r", [(16, 16, 8), (64, 32, 8), (128, 96, 16), (2048, 2048, 16), (144, 80, 24), (48, 272, 40),
                                   (2880, 2880, 16), (1040, 528, 64), (512, 1536, 128), (4112, 64, 120), (80, 4112, 32)])
@pytest.mark.parametrize("T", [1, 5])
def test_single_tokens(T, K, N, r):
    Case(T, K, N, r, 3, [(2 - i) % 3 for i in range(T)]).run().check()


@pytest.mark.parametrize("T", [2, 64, 200, 300])
def test_many_single_tokens(T):
    Case(T, 256, 320, 16, 11, [(7 * i) % 12 - 1 for i in range(T)]).run().check()


@pytest.mark.parametrize("T,K,N,r", [(16, 2048, 4112, 16), (80, 2064, 8208, 24), (150, 4096, 4112, 64), (320, 1024, 4112, 128),
                                     (300, 2048, 8192, 8)])
def test_single_tokens_over_many_buffers(T, K, N, r):
    """Every cluster size (8, 4, 2 and 1), more chunks than buffers, several passes over the columns."""
    Case(T, K, N, r, 5, [i % 6 - 1 for i in range(T)]).run().check()


@pytest.mark.parametrize("lens", [[1], [2], [8], [9], [15, 1], [127], [128], [129], [1, 1, 1], [0, 0, 3], [60, 1, 0, 200, 7],
                                  [16, 16, 16, 16], [65], [33, 1, 31, 8], [16] * 6, [1] * 20 + [50], [1] * 140,
                                  [300, 1, 1, 1, 500], [1] * 40 + [100]])
@pytest.mark.parametrize("K,N,r", [(64, 48, 8), (320, 400, 16), (144, 656, 64)])
def test_packed_requests(lens, K, N, r):
    off = np.cumsum([0] + lens).tolist()
    ad = [(5 * i) % 4 - (i % 3 == 2) for i in range(len(lens))]
    Case(off[-1], K, N, r, 4, ad, off, seed=len(lens)).run().check()


@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 48, 64, 72, 96, 120, 128])
def test_ranks(r):
    off = [0, 150, 151, 290]
    Case(300, 272, 336, r, 2, [1, 0, 1], off).run().check()


@pytest.mark.parametrize("lead", [0, 3])
def test_rows_of_no_request_stay(lead):
    off = [lead, 40, 40, 170, 200]
    Case(260, 96, 112, 16, 3, [2, 0, -1, 1], off).run().check()


@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("ldx,ldy", [(8, 0), (0, 24), (16, 40)])
def test_strided_rows(single, ldx, ldy):
    T = 30 if single else 210
    off = None if single else [0, 5, 200]
    ad = [i % 3 - 1 for i in range(T)] if single else [1, 0]
    Case(T, 160, 144, 16, 2, ad, off, ldx=ldx, ldy=ldy).run().check()


@pytest.mark.parametrize("off", [None, [0, 5, 150]])
@pytest.mark.parametrize("first", ["X", "Y"])
def test_rows_side_by_side_in_one_buffer(off, first):
    """X and Y as columns of one buffer, with columns between and behind them that stay."""
    T, K, N = (20 if off is None else 150), 96, 80
    ad = [i % 2 for i in range(T if off is None else 2)]
    c = Case(T, K, N, 16, 2, ad, off)
    buf = torch.randn(T, K + N + 24).to(BF).cuda()
    x0, y0 = (0, K + 16) if first == "X" else (N + 16, 0)
    c.X, c.Y = buf[:, x0:x0 + K], buf[:, y0:y0 + N]
    c.Ys, c.ldy = c.Y, 0
    start = buf.clone()
    c.run().check()
    rest = torch.ones(buf.shape[1], dtype=torch.bool)
    rest[y0:y0 + N] = False
    assert torch.equal(buf[:, rest.cuda()], start[:, rest.cuda()])


def test_long_and_wide():
    Case(3000, 2048, 1536, 16, 4, [0, 3, 1], [0, 1100, 1101, 2990]).run().check()
    Case(700, 7168, 2048, 32, 2, [1, 0], [0, 350, 700]).run().check()


@pytest.mark.parametrize("T,K,N,r", [(140, 1024, 528, 128), (140, 2880, 272, 40), (300, 576, 1040, 64), (300, 528, 64, 8),
                                     (5125, 1024, 64, 16), (5125, 256, 144, 72), (12800, 512, 64, 32), (25700, 128, 48, 16)])
def test_tiles_over_clusters_of_every_size(T, K, N, r):
    cut = T // 2 - 7
    Case(T, K, N, r, 3, [2, 0, 1], [0, cut, cut + 1, T - 3]).run().check()


def test_many_packed_requests():
    """More requests than a block has threads, most of them short, beside prompts."""
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 4, (400,), generator=g).tolist()
    lens[3], lens[170], lens[399] = 700, 900, 260
    off = np.cumsum([2] + lens).tolist()
    Case(off[-1] + 3, 192, 144, 16, 5, [i % 6 - 1 for i in range(400)], off).run().check()


def test_rows_past_32_bits():
    """Rows of Y (and of X) that begin past 2^31 elements."""
    ld, T = 4096, (1 << 19) + 300
    Y = torch.zeros(T, ld, dtype=BF, device="cuda")
    X = torch.zeros(T, ld, dtype=BF, device="cuda")
    A, B = torch.ones(1, 64, 8, dtype=BF, device="cuda"), torch.ones(1, 8, 32, dtype=BF, device="cuda")
    X[-200:, :64] = 0.5
    scale = torch.ones(1, device="cuda")
    idx = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")      # noqa: E731
    for off, ad in (([0, T - 200, T], [-1, 0]), ([0, T - 3, T], [-1, 0]), (None, None)):
        if off is None:
            ad = torch.full((T,), -1, dtype=torch.int32, device="cuda")
            ad[-3:] = 0
        else:
            ad = idx(ad)
        Y.zero_()
        ml.moe_lora_requests(X[:, :64], ad, A, B, scale, Y[:, :32], None if off is None else idx(off))
        n = 200 if off is not None and off[1] == T - 200 else 3
        assert torch.equal(Y[-n:, :32], torch.full((n, 32), 256.0, dtype=BF, device="cuda"))
        assert not Y[:-n].any() and not Y[-n:, 32:].any()
    assert ml.moe_get_device_error() == ml.MOE_OK


def test_not_finite_rows_keep_to_themselves():
    for off, ad in (([0, 200], [0]), (None, [0] * 200)):
        c = Case(200, 128, 96, 16, 1, ad, off)
        want = Case(200, 128, 96, 16, 1, ad, off).run()
        c.Xs[17, 3], c.Xs[90, 5], c.Ys[40, 7] = float("nan"), float("inf"), float("inf")
        c.run()
        rest = [i for i in range(200) if i not in (17, 90, 40)]
        assert torch.equal(c.Y[rest], want.Y[rest])
        assert torch.isnan(c.Y[17]).all() and not torch.isfinite(c.Y[90]).any() and torch.isinf(c.Y[40, 7])
        assert torch.isfinite(c.Y[40]).sum() == 95
    # rows without an adapter may hold anything
    c = Case(20, 64, 64, 8, 1, [0, -1], [0, 10, 20])
    c.Xs[10:] = float("nan")
    c.run()
    assert torch.isfinite(c.Y).all()


def test_bad_adapters_and_offsets_are_reported():
    for off, ad in (([0, 10, 40], [0, 3]), (None, [0] * 39 + [3]), ([0, 30, 20, 40], [0, 1, 2]), ([0, 20, 41], [0, 1]),
                    ([-5, 20, 40], [0, 1])):
        c = Case(40, 64, 64, 8, 3, ad, off)
        with pytest.raises(AssertionError):
            c.run()
        assert ml.moe_get_device_error() == ml.MOE_OK
    # offsets that decrease by more than a window, so that requests claim the same rows
    for off in ([0, 300, 100, 400], [0, 390, 10, 20, 380, 400], [0] + [400, 0] * 40 + [400]):
        c = Case(400, 1024, 64, 8, 3, [i % 3 for i in range(len(off) - 1)], off)
        with pytest.raises(AssertionError):
            c.run()
        assert ml.moe_get_device_error() == ml.MOE_OK
    c = Case(40, 64, 64, 8, 3, [0, 3], [0, 10, 40])
    before = c.Y.clone()
    c.call()
    torch.cuda.synchronize()
    assert ml.moe_get_device_error() == ml.MOE_ERR_DEVICE_INDEX
    assert torch.equal(c.Y[10:], before[10:])


def test_no_rows_and_no_adapters():
    Case(0, 64, 64, 8, 2, []).run()
    Case(0, 64, 64, 8, 2, [1, 0], [0, 0, 0]).run()
    Case(9, 64, 64, 8, 0, [-1] * 9).run().check()


@pytest.mark.parametrize("off", [None, [0, 1, 150, 151, 280, 300]])
def test_repeatable_on_streams_and_in_a_graph(off):
    ad = [i % 4 - 1 for i in range(300)] if off is None else [0, 1, 2, -1, 0]
    make = lambda: Case(300, 512, 640, 16, 3, ad, off, seed=2)      # noqa: E731
    want = make().run().Y
    assert torch.equal(make().run().Y, want)
    c = make()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c.call(st)
    st.synchronize()
    assert torch.equal(c.Y, want)
    c = make()
    start = c.Ys.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    for _ in range(2):
        c.Ys.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.Y, want)


def test_two_calls_on_two_streams():
    a = Case(500, 256, 512, 16, 3, [0, 1, 2], [0, 100, 300, 500], seed=1)
    b = Case(64, 256, 512, 32, 5, [i % 5 for i in range(64)], seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for c in (a, b):
        c.before = c.Ys.clone()
    torch.cuda.synchronize()
    a.call(s1)
    b.call(s2)
    torch.cuda.synchronize()
    assert ml.moe_get_device_error() == ml.MOE_OK
    a.check()
    b.check()


def test_refusals():
    z = lambda *s, t=BF: torch.zeros(*s, dtype=t, device="cuda")      # noqa: E731
    ad, c = z(4, t=torch.int32), z(2, t=torch.float32)
    ok = dict(X=z(4, 64), adapters=ad, A=z(2, 64, 8), B=z(2, 8, 32), scale=c, Y=z(4, 32))
    ml.moe_lora_requests(**ok)
    for kw in (dict(X=z(4, 64, t=torch.float16)), dict(A=z(2, 48, 8)), dict(B=z(2, 16, 32)), dict(B=z(3, 8, 32)),
               dict(scale=z(2)), dict(Y=z(5, 32)), dict(adapters=z(3, t=torch.int32)), dict(adapters=z(4, t=torch.int64)),
               dict(X=z(64, 4).t()), dict(A=z(2, 8, 64).transpose(1, 2)), dict(seq_offsets=ad)):
        with pytest.raises(ValueError):
            ml.moe_lora_requests(**{**ok, **kw})
    for kw in (dict(X=z(4, 66)[:, 2:]), dict(Y=z(4, 36)[:, :32]), dict(A=z(2, 64, 12), B=z(2, 12, 32))):
        with pytest.raises(ml.MoEError):
            ml.moe_lora_requests(**{**ok, **kw})


@pytest.mark.parametrize("K,N,r,lens", [(64, 8208, 16, [45, 90, 77, 1, 130]), (192, 4112, 32, [33, 31, 95, 200, 14]),
                                        (128, 4112, 128, [130, 50, 100]), (2048, 4096, 64, [100, 300, 259])])
def test_ragged_edges_over_many_column_stages(K, N, r, lens):
    """Every request begins and ends inside a box of rows, whose slots are used again and again: every
    run gives the same bits."""
    off = np.cumsum([3] + lens).tolist()
    make = lambda: Case(off[-1] + 5, K, N, r, 3, [i % 3 for i in range(len(lens))], off, seed=K)      # noqa: E731
    want = make().run()
    want.check()
    for _ in range(8):
        assert torch.equal(make().run().Y, want.Y)


@pytest.mark.parametrize("tiles,K,r", [(148, 16384, 64), (296, 16384, 16), (148, 16384, 128), (1, 65536, 32)])
def test_long_sums_keep_their_digits(tiles, K, r):
    """X A over many columns, all of one sign, B the identity and Y the negative of the rounded result,
    so that Y ends as what the rounding left, a few digits of which show the sum's own error.

    Bound, of the sum: an instruction adds 16 products to an accumulator and cuts off less than a unit
    in its last place, 2^-23, at most twice (aligning the summands, and the result).  A sum runs through
    2 accumulators or more, K / 32 instructions; at ranks up to 64 through 4, K / 64.  Four fp32 additions
    and the scale, 2^-24 each; c X A as two bf16, 2^-17; and Y's own rounding, 2^-8 of what is left."""
    T, N = 128 * tiles, 16 * ((r + 15) // 16)
    g = torch.Generator(device="cuda").manual_seed(K + r)
    X = torch.randn(T, K, generator=g, device="cuda").to(BF).abs_()
    A = torch.randn(1, K, r, generator=g, device="cuda").to(BF).abs_()
    B = torch.zeros(1, r, N, device="cuda")
    B[0, :, :r] = torch.eye(r, device="cuda")
    ref = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for i in range(0, T, 2048):
        ref[i:i + 2048, :r] = X[i:i + 2048].double() @ A[0].double()
    Y = -ref.to(BF)
    want = Y.double() + ref
    ml.moe_lora_requests(X, torch.zeros(1, dtype=torch.int32, device="cuda"), A, B.to(BF), torch.ones(1, device="cuda"),
                         Y, torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert ml.moe_get_device_error() == ml.MOE_OK
    chain = K / (32 if r > 64 else 64)
    tol = (chain * 2.0 ** -22 + 5 * U + 2.0 ** -17) * ref + 2.0 ** -8 * want.abs()
    assert ((Y.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("r", [8, 16, 24, 40, 64, 72])
@pytest.mark.parametrize("off", [None, [0, 140, 200]])
def test_infinite_rows_follow_the_definition(off, r):
    """An infinity in X times positive adapters is an infinity in every entry, whatever the rank."""
    c = Case(200, 256, 96, r, 1, [0] * (200 if off is None else 2), off)
    c.A.abs_()
    c.B.abs_()
    c.Xs[17, 3], c.Xs[150, 200] = float("inf"), -float("inf")
    c.run()
    assert (c.Y[17] == float("inf")).all() and (c.Y[150] == -float("inf")).all()
    rest = [i for i in range(200) if i not in (17, 150)]
    assert torch.isfinite(c.Y[rest]).all()


@pytest.mark.parametrize("K,N,r", [(64, 528, 32), (64, 528, 24), (48, 528, 128), (64, 272, 72), (32, 1040, 16), (64, 784, 64)])
def test_tiles_without_a_cluster(K, N, r):
    """Up to 64 columns of X a tile is one CTA's, at every padded rank; the columns of Y run through its
    buffers more than once."""
    Case(300, K, N, r, 3, [2, 0, 1], [0, 143, 144, 297]).run().check()
