"""Paged cache on the GPU: rotated appends (16-bit, and E4M3 with a scale for each
page and KV head) and the single-token sink attention over them, against the
float64 oracle on the same rounded inputs.

Tolerances, from the arithmetic:
- a 16-bit result is rounded once: eps/2 of its value (plus half the smallest
  subnormal step of float16, 2^-25), after float32 products and sums whose error
  is under 2^-22 of the operands' magnitudes;
- an 8-bit element is off by at most 2^-4 of its value, or half the smallest
  step, 2^-10 of the block's scale, with the same float32 error;
- attention: a score of D <= 128 float32 products has an error under
  (D + 3) 2^-24 sum|q k| scale, at most 7e-5 for the normal draws here (sum|q k|
  scale < 9), so a weight is off by less than 2^-12.7 of itself; the weights'
  rounding on the tensor cores adds at most 2^-11 of a weight (and weights below
  2^-25 of the largest may be dropped).  The output is off by under
  2^-10 max|v|, plus its own rounding; LSE and the gate by under 2^-12.
"""
import threading

import numpy as np
import pytest
import torch

import oracle
from learnable_sink_b200 import sinkattn as S

from gpu_util import check_lse, check_status, np64

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TINY = {BF: 0.0, F16: 2.0 ** -25}


@pytest.fixture(autouse=True)
def _status():
    S.clear_status()
    yield
    check_status()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def make_table(lens, page, g, spare=2, width=None):
    width = width or max(1, -(-max(max(lens), 1) // page))
    n = len(lens) * width + spare
    return torch.randperm(n, generator=g)[: len(lens) * width].view(len(lens), width).int(), n


def make_pool(n_pages, Hkv, page, D, dtype, g, std=1.0):
    """(pages, scale or None): normal values, or their E4M3 codes (uint8)."""
    x = torch.randn(n_pages, Hkv, page, D, generator=g) * std
    if dtype is not None:
        return x.to(dtype), None
    scale = torch.exp2(torch.randint(-9, -4, (n_pages, Hkv), generator=g).float())
    codes = (x / scale[:, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), scale


class Problem:
    """A decode problem on the CPU; run() gives the GPU's results, want() the oracle's."""

    def __init__(self, lens, Hq, Hkv, D, page, dtype=BF, fp8=False, n_sink=0, window=0, sink=True,
                 seed=1, width=None):
        g = gen(seed)
        self.lens, self.dtype, self.fp8 = torch.tensor(lens, dtype=torch.int32), dtype, fp8
        self.n_sink, self.window = n_sink, window
        self.table, n = make_table(lens, page, g, width=width)
        pool = None if fp8 else dtype
        self.k, self.ks = make_pool(n, Hkv, page, D, pool, g)
        self.v, self.vs = make_pool(n, Hkv, page, D, pool, g)
        self.q = torch.randn(len(lens), Hq, D, generator=g).to(dtype)
        self.sink = torch.randn(Hq, generator=g) if sink else None
        self.scale = D ** -0.5

    def cache(self):
        f = lambda t: None if t is None else t.cuda()  # noqa: E731
        return S.PagedCache(f(self.k), f(self.v), f(self.table), f(self.lens), f(self.ks), f(self.vs))

    def run(self, cache=None, **kw):
        call = S.paged_decode_fp8 if self.fp8 else S.paged_decode
        out = call(self.q.cuda(), cache or self.cache(), None if self.sink is None else self.sink.cuda(),
                   n_sink=self.n_sink, window=self.window, scale=self.scale, **kw)
        torch.cuda.synchronize()
        return out

    def want(self):
        return oracle.paged_decode(self.q, self.k, self.v, self.table, self.lens, self.n_sink,
                                   self.window, self.sink, self.scale, self.ks, self.vs)

    def check(self, got=None, want=None, vmax=None):
        out, lse, ss = self.run() if got is None else got
        ro, rl, rs = self.want() if want is None else want
        vmax = 5.0 if vmax is None else vmax  # of the normal draws
        tol = torch.finfo(self.dtype).eps / 2 * np.abs(ro) + 2.0 ** -10 * vmax + TINY[self.dtype]
        d = np.abs(np64(out) - ro)
        assert (d <= tol).all(), (float(d.max()), float((d / tol).max()))
        check_lse(np64(lse), rl, 2.0 ** -12)
        assert np.abs(np64(ss) - rs).max() <= 2.0 ** -12


MIXED = [0, 1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 700]
KINDS = [(BF, False), (F16, False), (BF, True), (F16, True)]


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("dtype,fp8", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_lengths_and_pages(dtype, fp8, page, D):
    Problem(MIXED, 8, 2, D, page, dtype, fp8, seed=page + D).check()


@pytest.mark.parametrize("dtype,fp8", KINDS)
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 9, 16])
def test_decode_group_sizes(dtype, fp8, G):
    for D, Hkv in ((64, 3), (128, 1)):
        Problem([300, 5, 0, 129], G * Hkv, Hkv, D, 32, dtype, fp8, seed=G).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_sink,window", [(4, 60), (0, 1), (20, 130), (4, 5000), (300, 7), (1, 128),
                                           (0, 257), (128, 128)])
def test_decode_window_and_sink_tokens(fp8, n_sink, window):
    for page, D in ((16, 128), (64, 64)):
        Problem(MIXED + [1500], 8, 2, D, page, BF, fp8, n_sink, window, seed=window).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_without_a_sink(fp8):
    Problem(MIXED, 4, 2, 128, 16, BF, fp8, sink=False).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_long_and_unequal(fp8):
    """Work split over many blocks and joined again, next to single rows."""
    Problem([40000, 3, 9001, 128, 0, 257], 8, 2, 128, 64, BF, fp8, seed=5).check()
    Problem([33333], 4, 1, 64, 16, F16, fp8, seed=6).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_many_short_sequences(fp8):
    lens = torch.randint(0, 90, (1500,), generator=gen(7)).tolist()
    Problem(lens, 4, 2, 64, 16, BF, fp8, seed=8).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B", [128, 129])
def test_decode_many_split_sequences(fp8, B):
    """The join finds a pair's segments from the lengths, or with more sequences than it
    has threads from the decode kernel's note: lengths of which most pairs are cut."""
    lens = torch.randint(0, 900, (B,), generator=gen(55)).tolist()
    lens[3], lens[B - 1] = 0, 5000
    Problem(lens, 6, 3, 64, 32, BF, fp8, seed=56).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hkv", [5, 9, 10, 11, 16])
def test_decode_head_groups(fp8, Hkv):
    """Heads that one group of blocks covers, several do, or that share no divisor with a
    group: rows cut, rows of one length left whole, and more sequences than the join
    adds up for itself."""
    Problem([3000, 0, 1, 700, 2500], Hkv, Hkv, 64, 16, BF, fp8, seed=57).check()
    Problem([600, 590, 600], 2 * Hkv, Hkv, 128, 32, BF, fp8, seed=58).check()
    if Hkv == 10:
        lens = torch.randint(0, 500, (129,), generator=gen(59)).tolist()
        Problem(lens, Hkv, Hkv, 64, 64, BF, fp8, seed=60).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_decode_ignores_what_masked_rows_hold(fp8, bad):
    """Rows past the length, rows that the window hides, other pages and their
    scales hold NaN or infinities."""
    for n_sink, window in ((0, 0), (5, 40), (0, 129)):
        p = Problem([1, 40, 130, 300, 0], 8, 2, 128, 16, F16, fp8, n_sink, window, seed=9)
        want = p.want()
        used = torch.zeros(p.k.shape[0], p.k.shape[2], dtype=torch.bool)
        for b, n in enumerate(p.lens.tolist()):
            for j in range(n):
                if window == 0 or j < n_sink or j >= n - window:
                    used[p.table[b, j // 16], j % 16] = True
        hide = ~used[:, None, :, None].expand_as(p.k)
        value = float(bad)
        for pages in (p.k, p.v):
            if fp8:
                pages[hide] = 0x7F if bad == "nan" else 0xFE
            else:
                pages[hide] = value
        if fp8:
            unread = ~used.any(1)
            p.ks[unread] = value
            p.vs[unread] = value
        p.check(want=want)


@pytest.mark.parametrize("dtype,fp8", KINDS)
@pytest.mark.parametrize("slope", [9.0, 20.0, -9.0])
def test_decode_growing_scores(dtype, fp8, slope):
    """Scores that rise (or fall) by `slope` log2 units a 128 positions, so that
    the running maximum keeps moving."""
    p = Problem([900, 2000], 4, 2, 64, 64, dtype, fp8, seed=11)
    p.q.zero_()
    p.q[:, :, 0] = 8.0
    if fp8:
        p.ks.fill_(2.0 ** -2)
    for b, n in enumerate(p.lens.tolist()):
        for j in range(n):
            x = slope * (j - n / 2) / 128 * np.log(2.0) / (8.0 * p.scale)
            at = p.table[b, j // 64]
            p.k[at, :, j % 64] = 0
            if fp8:
                x = torch.tensor(x * 4).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            p.k[at, :, j % 64, 0] = x
    p.check()


@pytest.mark.parametrize("dtype,fp8", KINDS)
def test_decode_dominant_first_token(dtype, fp8):
    """An attention sink in the cache: the first token takes most of the weight,
    tens of thousands of others share the rest at about 2^-20 of it each.  With
    values 0 in the first token and 1 elsewhere the output is the others' share,
    which must not be lost (each weight is within 2^-8 of itself here, and the
    shares add up without cancelling)."""
    n = 50000
    p = Problem([n], 4, 1, 64, 128, dtype, fp8, sink=False, seed=12)
    p.q.zero_()
    p.q[:, :, 0] = 8.0
    one = 0x38 if fp8 else 1.0  # the code of 1
    if fp8:
        p.ks.fill_(1.0)
        p.vs.fill_(1.0)
    p.k.zero_()
    p.v.fill_(one)
    first = p.table[0, 0]
    p.k[first, :, 0, 0] = 0x56 if fp8 else 14.0  # the code of 14: a score of 14 = 20.2 log2 units
    p.v[first, :, 0] = 0
    want = p.want()
    out = p.run()[0]
    assert np.abs(np64(out) / want[0] - 1).max() <= 2.0 ** -7, (np64(out).max(), want[0].max())
    p.check(want=want, vmax=1.0)


def test_decode_scales_of_very_different_size():
    """Value scales from 2^-40 to 2^12 and blocks of zeros (scale 0): the result is
    held against its own largest term."""
    p = Problem([500, 90], 8, 2, 128, 16, BF, True, seed=13)
    p.vs = torch.exp2(torch.randint(-40, 13, p.vs.shape, generator=gen(14)).float())
    p.vs[::7] = 0
    p.ks[::5] = 0
    for b in range(2):  # a sequence whose values are all tiny
        if b == 1:
            p.vs[p.table[b].long()] *= 2.0 ** -40
    want = p.want()
    out, lse, ss = p.run()
    val = oracle.fp8_e4m3_value(p.v.numpy()) * p.vs.double().numpy()[:, :, None, None]
    for b in range(2):
        top = np.abs(val[p.table[b].numpy()]).max()
        d = np.abs(np64(out[b]) - want[0][b])
        assert (d <= 2.0 ** -9 * np.abs(want[0][b]) + 2.0 ** -10 * top).all()
    check_lse(np64(lse), want[1], 2.0 ** -12)
    assert np.abs(np64(ss) - want[2]).max() <= 2.0 ** -12


def test_decode_any_scale_and_one_sequence_at_the_end_of_the_range():
    """Scales need not be powers of two; an infinite sink logit of either sign."""
    p = Problem([200, 31], 8, 2, 128, 32, BF, True, seed=15)
    p.ks *= torch.rand(p.ks.shape, generator=gen(16)) + 0.5
    p.vs *= torch.rand(p.vs.shape, generator=gen(17)) + 0.5
    p.check()
    p.sink[0] = -np.inf
    p.sink[5] = 80.0
    p.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_nan_in_a_visible_row_reaches_the_output(fp8):
    p = Problem([100, 100], 4, 2, 64, 16, BF, fp8, seed=18)
    at = p.table[0, 3]
    p.k[at, 1, 5, 7] = 0x7F if fp8 else float("nan")
    want = Problem([100, 100], 4, 2, 64, 16, BF, fp8, seed=18).want()
    out, lse, _ = p.run()
    assert torch.isnan(out[0, 2:]).all() and torch.isnan(lse[0, 2:]).all()
    p.check(got=(out[1:], lse[1:], _[1:]), want=[w[1:] for w in want])
    p = Problem([100, 100], 4, 2, 64, 16, BF, fp8, seed=18)
    p.v[at, 1, 5, 7] = 0x7F if fp8 else float("nan")
    out, lse, _ = p.run()
    assert torch.isnan(out[0, 2:, 7]).all()
    assert not torch.isnan(out[0, :2]).any() and not torch.isnan(out[1]).any()
    check_lse(np64(lse), want[1], 2.0 ** -12)


@pytest.mark.parametrize("dtype", [BF, F16])
def test_decode_infinity_in_a_visible_row(dtype):
    """A value's reaches its own element of its heads, not as a finite number; a key's
    takes all of the weight or none."""
    clean = Problem([300, 100], 4, 2, 64, 16, dtype, seed=51)
    want = clean.want()
    p = Problem([300, 100], 4, 2, 64, 16, dtype, seed=51)
    at = p.table[0, 3]
    p.v[at, 1, 5, 7] = float("inf")
    out, lse, ss = p.run()
    assert not torch.isfinite(out[0, 2:, 7]).any()
    out[0, 2:, 7] = torch.from_numpy(want[0][0, 2:, 7]).to(out)
    p.check((out, lse, ss), want)
    # scores of -inf: the row is as if it were masked; of +inf: NaN, as e^{inf - inf} is
    p = Problem([300, 100], 4, 2, 64, 16, dtype, seed=51)
    p.k[at, 1, 5, 7] = float("inf")
    p.q[0, 2, 7], p.q[0, 3, 7] = -1.0, 1.0
    out, lse, ss = p.run()
    assert torch.isnan(out[0, 3]).all() and torch.isnan(lse[0, 3])
    p.k[at, 1, 5, 7] = 0.0
    p.k[at, 1, 5] = -256.0 * torch.sign(p.q[0, 2].float()).to(dtype)  # a score below -200
    want = p.want()
    rows = lambda a: np.concatenate([a[0, :3], a[1]])  # noqa: E731
    p.check([torch.from_numpy(rows(np64(t))) for t in (out, lse, ss)], [rows(w) for w in want])


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_shared_prefix_pages(fp8):
    """Several sequences read the same pages."""
    p = Problem([500, 450, 500], 8, 2, 128, 32, BF, fp8, seed=19)
    p.table[1, :12] = p.table[0, :12]
    p.table[2] = p.table[0]
    p.q[2] = p.q[0]
    got = p.run()
    p.check(got)
    # The third sequence equals the first, but its work may be cut elsewhere, which orders
    # the sums differently: a weight is off by 2^-22 (the exponential) and 2^-21 (its
    # argument, below 16 in log2 units), a sum of them by some 20 additions' 2^-24 each;
    # together under 2^-18.  LSE and the gate round once more, below 2^-20.
    assert all((t[0] - t[2]).abs().max() <= 2.0 ** -17 for t in got[1:])


def test_decode_bad_pages_and_lengths_set_the_status():
    """Table entries outside the pool are skipped like masked rows, a length past
    the table counts as the table's; both set SINKATTN_ERR_BOUNDS."""
    for fp8 in (False, True):
        for bad in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
            p = Problem([100, 60], 4, 2, 128, 16, BF, fp8, seed=20)
            ref = Problem([100, 60], 4, 2, 128, 16, BF, fp8, 16, 68, seed=20)  # rows [16, 32) hidden
            want = ref.want()
            p.table[0, 1] = bad
            out = p.run()
            assert S.get_status() == 6
            S.clear_status()
            p.check(out, want=[np.concatenate([w[:1], x[1:]]) for w, x in
                               zip(want, Problem([100, 60], 4, 2, 128, 16, BF, fp8, seed=20).want())])
        p = Problem([100, 60], 4, 2, 128, 16, BF, fp8, seed=21)
        want = Problem([112, 60], 4, 2, 128, 16, BF, fp8, seed=21).want()
        p.lens[0] = 2 ** 31 - 1
        out = p.run()
        assert S.get_status() == 6
        S.clear_status()
        p.check(out, want=want)
        p.lens[:] = torch.tensor([-5, -2 ** 31], dtype=torch.int32)
        out, lse, ss = p.run()
        assert (out == 0).all() and (ss == 0).all()
        # a goes through a log2(e) and ln(2) back: two products and two constants, each off
        # by at most 2^-24 of itself, so lse is within 4 2^-24 |a| (to first order) of a
        assert (lse.cpu() - p.sink).abs().le(2.0 ** -21.9 * p.sink.abs()).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_repeats_bitwise_with_any_workspace(fp8):
    p = Problem([5000, 1, 700, 129], 8, 2, 128, 64, BF, fp8, seed=22)
    c = p.cache()
    n = S.paged_decode_workspace_bytes(4, 8, 2, 128)
    first = p.run(c, workspace=torch.zeros(n, dtype=torch.uint8, device="cuda"))
    for fill in (0xFF, 0x7F):
        again = p.run(c, workspace=torch.full((n,), fill, dtype=torch.uint8, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    p.check(first)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_captured_with_lengths_that_change(fp8):
    """One captured call replayed while lengths, tables and queries change."""
    lens = [700, 30, 128]
    p = Problem(lens, 8, 2, 128, 32, BF, fp8, 4, 300, seed=23, width=40)
    c = p.cache()
    call = S.paged_decode_fp8 if fp8 else S.paged_decode
    q, sink = p.q.cuda(), p.sink.cuda()
    ws = torch.empty(S.paged_decode_workspace_bytes(3, 8, 2, 128), dtype=torch.uint8, device="cuda")
    kw = dict(n_sink=4, window=300, workspace=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(q, c, sink, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call(q, c, sink, **kw)
    for new in ([700, 30, 128], [1280, 0, 1], [3, 1000, 650]):
        p.lens[:] = torch.tensor(new, dtype=torch.int32)
        p.q = torch.randn(p.q.shape, generator=gen(sum(new))).to(BF)
        c.cache_seqlens.copy_(p.lens)
        q.copy_(p.q)
        g.replay()
        torch.cuda.synchronize()
        p.check(got)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_on_two_streams_at_once(fp8):
    """Calls that overlap on two streams, each with its own workspace."""
    ps = [Problem([3000, 20, 999], 8, 2, 128, 32, BF, fp8, seed=s) for s in (24, 25)]
    cs, qs, sinks = [p.cache() for p in ps], [p.q.cuda() for p in ps], [p.sink.cuda() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    call = S.paged_decode_fp8 if fp8 else S.paged_decode
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(call(qs[i], cs[i], sinks[i]))
    torch.cuda.synchronize()
    for p, runs in zip(ps, got):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))
        p.check(runs[0])


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_two_graphs_share_a_workspace(fp8):
    """Two captured calls of different shapes, replayed in turn over one workspace, and
    a call on a stream passed by argument."""
    ps = [Problem([2000, 9, 600], 8, 2, 128, 64, BF, fp8, seed=27), Problem([50, 1300], 16, 2, 128, 64, BF, fp8, seed=28)]
    ws = torch.empty(max(S.paged_decode_workspace_bytes(3, 8, 2, 128),
                         S.paged_decode_workspace_bytes(2, 16, 2, 128)), dtype=torch.uint8, device="cuda")
    call = S.paged_decode_fp8 if fp8 else S.paged_decode
    graphs, outs, held = [], [], []
    for p in ps:
        q, c, sink = p.q.cuda(), p.cache(), p.sink.cuda()
        held.append((q, c, sink))
        call(q, c, sink, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(q, c, sink, workspace=ws))
        graphs.append(g)
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for p, o in zip(ps, outs):
        p.check(o)
    side = torch.cuda.Stream()
    ps[0].check(ps[0].run(stream=side))


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_back_to_back_without_a_wait(fp8):
    """Many calls in a row whose inputs the stream itself changes in between: each
    starts under the end of the one before it, and none may read too early."""
    p = Problem([700, 1, 129, 40], 8, 2, 64, 16, BF, fp8, seed=29)
    c, sink = p.cache(), p.sink.cuda()
    qs = [torch.randn(p.q.shape, generator=gen(100 + i)).to(BF) for i in range(12)]
    lens = [torch.tensor([700 - 31 * i, i, 129 - 7 * i, 40 + i], dtype=torch.int32) for i in range(12)]
    qd, ld = [x.cuda() for x in qs], [x.cuda() for x in lens]
    q = torch.empty_like(qd[0])
    call = S.paged_decode_fp8 if fp8 else S.paged_decode
    ws = torch.empty(S.paged_decode_workspace_bytes(4, 8, 2, 64), dtype=torch.uint8, device="cuda")
    got = []
    torch.cuda.synchronize()
    for i in range(12):
        q.copy_(qd[i])
        c.cache_seqlens.copy_(ld[i])
        got.append(call(q, c, sink, workspace=ws))
        got.append(call(q, c, sink, workspace=ws))  # the call before it is the same kernel
    torch.cuda.synchronize()
    for i in range(12):
        p.q, p.lens = qs[i], lens[i]
        want = p.want()
        p.check(got[2 * i], want)
        p.check(got[2 * i + 1], want)


def test_decode_row_offsets_past_32_bits():
    """Pages whose element offsets pass 2^31."""
    page, D, Hkv = 128, 128, 1
    n = (1 << 31) // (page * D) + 40
    g = gen(26)
    p = Problem([300, 500], 4, 1, D, page, BF, True, seed=26)
    high = torch.randperm(36, generator=g)[: p.table.numel()].view_as(p.table).int() + (n - 40)
    small = {int(a): int(b) for a, b in zip(p.table.flatten(), high.flatten())}
    pools = []
    for t in (p.k, p.v):
        big = torch.zeros(n, Hkv, page, D, dtype=torch.uint8, device="cuda")
        for a, b in small.items():
            big[b] = t[a].cuda()
        pools.append(big)
    scales = []
    for t in (p.ks, p.vs):
        big = torch.ones(n, Hkv, device="cuda")
        for a, b in small.items():
            big[b] = t[a].cuda()
        scales.append(big)
    c = S.PagedCache(pools[0], pools[1], high.cuda(), p.lens.cuda(), *scales)
    p.check(p.run(c))
    # the append writes there, too
    x = torch.randn(2, Hkv, D, generator=g).to(BF)
    S.paged_append_fp8(x.cuda(), x.cuda(), c)
    torch.cuda.synchronize()
    want, ws = oracle.paged_append_fp8(x, p.table, p.lens, p.k, p.ks)
    for b, m in enumerate(p.lens.tolist()):
        a = int(p.table[b, (m - 1) // page])
        assert torch.equal(pools[0][small[a]].cpu(), torch.from_numpy(want[a]))
        assert float(scales[0][small[a], 0]) == ws[a, 0]


# ------------------------------------------------------------------ append
def append_case(new, past, Hq, Hkv, D, page, dtype, rot, seed, fp8):
    """Packed tokens (views of one projection's output), a cache and its lengths."""
    g = gen(seed)
    lens = [a + b for a, b in zip(new, past)]
    T = sum(new)
    x = torch.randn(T + 2, Hq + 2 * Hkv, D, generator=g).to(dtype)  # two rows behind the last
    table, n = make_table(lens, page, g)
    pool = None if fp8 else dtype
    k, ks = make_pool(n, Hkv, page, D, pool, g)
    v, vs = make_pool(n, Hkv, page, D, pool, g)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    rope = None if rot is None else torch.from_numpy(oracle.rope_table(max(max(lens), 1), rot)).float()
    return dict(x=x, T=T, cu=cu, table=table, lens=torch.tensor(lens, dtype=torch.int32), k=k, v=v,
                ks=ks, vs=vs, rope=rope)


def positions(c, single=False):
    cu, lens = c["cu"].tolist(), c["lens"].tolist()
    pos = np.zeros(c["x"].shape[0], dtype=np.int64)
    for b, n in enumerate(lens):
        for t in range(cu[b], cu[b + 1]):
            pos[t] = n - (cu[b + 1] - t)
    return pos


def near16(got, want, mag, dtype):
    tol = torch.finfo(dtype).eps / 2 * np.abs(want) + 2.0 ** -22 * mag + TINY[dtype]
    d = np.abs(got - want)
    assert (d <= tol * (1 + 1e-9)).all(), float((d / np.maximum(tol, 1e-300)).max())


NEW = [0, 1, 2, 17, 5, 130, 16, 0]
PAST = [3, 0, 15, 20, 64, 7, 16, 0]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("D,page,rot,inter", [(128, 16, 128, False), (128, 64, 64, True),
                                              (64, 32, 16, False), (64, 128, 64, True),
                                              (128, 32, 48, False), (64, 16, None, False)])
def test_append_rotates_and_places(dtype, D, page, rot, inter):
    """Every row of every page, the rotated queries and keys, and the rows behind the
    last sequence, which stay as they were."""
    Hq, Hkv = 8, 2
    c = append_case(NEW, PAST, Hq, Hkv, D, page, dtype, rot, D + page, False)
    x = c["x"].cuda()
    T = x.shape[0]
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cache = S.PagedCache(c["k"].cuda(), c["v"].cuda(), c["table"].cuda(), c["lens"].cuda())
    q_out = torch.full((T, Hq, D), 7.0, dtype=dtype, device="cuda")
    k_out = torch.full((T, Hkv, D), 7.0, dtype=dtype, device="cuda")
    r = S.paged_append(k, v, cache, c["cu"].cuda(), None if rot is None else c["rope"].cuda(), inter,
                       q=q, q_out=q_out, k_out=k_out)
    torch.cuda.synchronize()
    assert r is q_out and torch.equal(x.cpu(), c["x"])
    n = c["T"]
    X = c["x"].double().numpy()
    wq, wk = X[:, :Hq].copy(), X[:, Hq:Hq + Hkv].copy()
    if rot is not None:
        pos = positions(c)
        wq, wk = (oracle.rotate(t, pos, c["rope"], inter) for t in (wq, wk))
    near16(np64(q_out[:n]), wq[:n], 8.0, dtype)
    near16(np64(k_out[:n]), wk[:n], 8.0, dtype)
    assert (q_out[n:] == 7).all() and (k_out[n:] == 7).all()
    ep, ev = oracle.paged_append(np64(k_out), X[:, Hq + Hkv:], c["table"], c["lens"], c["k"], c["v"],
                                 c["cu"])
    assert np.array_equal(np64(cache.k_pages), ep)
    assert np.array_equal(np64(cache.v_pages), ev)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("D,page,rot,inter", [(128, 16, 128, False), (128, 64, 64, True),
                                              (64, 32, 16, False), (64, 128, 64, True),
                                              (128, 128, None, False), (64, 16, 64, False)])
def test_append_fp8_scales_and_codes(dtype, D, page, rot, inter):
    """Scales and re-encoded earlier rows exactly; new rows within half a step of the
    grid; everything else untouched.  Some new tokens are 30 times larger."""
    Hq, Hkv = 8, 2
    c = append_case(NEW, PAST, Hq, Hkv, D, page, dtype, rot, D + page + 1, True)
    c["x"][::5] *= 30
    c["x"][3, Hq] = 0
    x = c["x"].cuda()
    T = x.shape[0]
    cache = S.PagedCache(c["k"].cuda(), c["v"].cuda(), c["table"].cuda(), c["lens"].cuda(),
                         c["ks"].cuda(), c["vs"].cuda())
    q_out = torch.full((T, Hq, D), 7.0, dtype=dtype, device="cuda")
    k_out = torch.full((T, Hkv, D), 7.0, dtype=dtype, device="cuda")
    S.paged_append_fp8(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, c["cu"].cuda(),
                       None if rot is None else c["rope"].cuda(), inter, q=x[:, :Hq], q_out=q_out,
                       k_out=k_out)
    torch.cuda.synchronize()
    n, X = c["T"], c["x"].double().numpy()
    wq, wk, wv = X[:, :Hq].copy(), X[:, Hq:Hq + Hkv].copy(), X[:, Hq + Hkv:]
    pos = positions(c)
    if rot is not None:
        wq, wk = (oracle.rotate(t, pos, c["rope"], inter) for t in (wq, wk))
    near16(np64(q_out[:n]), wq[:n], 240.0, dtype)
    near16(np64(k_out[:n]), wk[:n], 240.0, dtype)
    assert (q_out[n:] == 7).all() and (k_out[n:] == 7).all()
    for val, codes0, sc0, codes, sc in ((wk, c["k"], c["ks"], cache.k_pages, cache.k_scale),
                                        (wv, c["v"], c["vs"], cache.v_pages, cache.v_scale)):
        want, ws = oracle.paged_append_fp8(val, c["table"], c["lens"], codes0, sc0, c["cu"])
        assert np.array_equal(np64(sc), ws)
        got = codes.cpu().numpy()
        fresh = np.zeros(got.shape[:1] + got.shape[2:3], dtype=bool)
        for t, b, p in oracle._new_tokens(c["cu"], c["lens"]):
            at = int(c["table"][b, p // page])
            fresh[at, p % page] = True
            s = ws[at][:, None]
            d = np.abs(oracle.fp8_e4m3_value(got[at, :, p % page]) * s - val[t])
            tol = np.maximum(2.0 ** -4 * np.abs(val[t]), 2.0 ** -10 * s) + 2.0 ** -22 * 240
            assert (d <= tol).all()
        keep = ~fresh[:, None, :, None].repeat(Hkv, 1).repeat(D, 3)
        assert np.array_equal(got[keep], want[keep])


@pytest.mark.parametrize("Hkv", [1, 3, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_append_fp8_heads_do_not_touch_each_other(D, Hkv):
    """Any number of heads gives each the bits that it gets alone, though blocks may hold
    two; heads differ in size, so a neighbour's scale would show."""
    page = 32
    c = append_case(NEW, PAST, 0, Hkv, D, page, BF, D, 54 + Hkv, True)
    c["x"] *= torch.exp2(torch.arange(2 * Hkv).float() * 3)[:, None].to(BF)
    x, rope, cu = c["x"].cuda(), c["rope"].cuda(), c["cu"].cuda()
    table, lens = c["table"].cuda(), c["lens"].cuda()

    def run(heads):
        pools = [c[n][:, heads].contiguous().cuda() for n in ("k", "v", "ks", "vs")]
        cache = S.PagedCache(pools[0], pools[1], table, lens, *pools[2:])
        k, v = x[:, :Hkv][:, heads].contiguous(), x[:, Hkv:][:, heads].contiguous()
        k_out = torch.zeros_like(k)
        S.paged_append_fp8(k, v, cache, cu, rope, k_out=k_out)
        torch.cuda.synchronize()
        return pools, k_out

    pools, k_out = run(slice(0, Hkv))
    for h in range(Hkv):
        alone, k_alone = run(slice(h, h + 1))
        assert all(torch.equal(a[:, h], b[:, 0]) for a, b in zip(pools, alone))
        assert torch.equal(k_out[:, h], k_alone[:, 0])


def test_append_fp8_special_values():
    """Infinities saturate and set no scale, NaN stays NaN, a block of zeros has
    scale 0 and grows later, tiny values take the smallest scale, and a value of
    exactly 448 s does not move the scale."""
    D, page = 64, 16
    x = torch.zeros(6, 1, D, dtype=BF)
    x[0, 0, :3] = torch.tensor([float("inf"), -float("inf"), 3.5])
    x[1, 0, 0] = float("nan")
    x[1, 0, 1] = 1.0
    x[3, 0, 0] = 2.0 ** -133
    x[4, 0, 0] = 3.0e38
    x[5, 0, 0] = 3.5 + 2.0 ** -6
    B = 6
    table = torch.arange(B).view(B, 1).int()
    lens = torch.ones(B, dtype=torch.int32)
    k = torch.full((B, 1, page, D), 0x11, dtype=torch.uint8)
    cache = S.PagedCache(k.cuda(), k.cuda(), table.cuda(), lens.cuda(),
                         torch.full((B, 1), 3.0).cuda(), torch.full((B, 1), 3.0).cuda())
    S.paged_append_fp8(x.cuda(), x.cuda(), cache)
    torch.cuda.synchronize()
    want, ws = oracle.paged_append_fp8(x, table, lens, k, torch.full((B, 1), 3.0))
    assert ws[:, 0].tolist() == [2.0 ** -7, 2.0 ** -8, 0.0, 2.0 ** -126, 2.0 ** 120, 2.0 ** -6]
    for codes, sc in ((cache.k_pages, cache.k_scale), (cache.v_pages, cache.v_scale)):
        assert np.array_equal(np64(sc), ws)
        assert np.array_equal(codes.cpu().numpy(), want)
    # the block of zeros takes a row that needs a scale
    y = torch.full((B, 1, D), 2.0, dtype=BF)
    cache.cache_seqlens.fill_(2)
    S.paged_append_fp8(y.cuda(), y.cuda(), cache)
    torch.cuda.synchronize()
    want, ws = oracle.paged_append_fp8(y, table, lens * 2, want, ws)
    assert np.array_equal(np64(cache.k_scale), ws)
    assert np.array_equal(cache.k_pages.cpu().numpy(), want)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_one_token_a_sequence(fp8):
    """Without cu_new; idle slots of a padded batch write nothing; q in place."""
    Hq, Hkv, D, page = 8, 2, 128, 16
    past = [0, 15, 16, 31, 100, 7]
    c = append_case([1] * 6, past, Hq, Hkv, D, page, BF, 128, 41, fp8)
    c["lens"][5] = 0
    x = c["x"][:6]
    f = lambda t: None if t is None else t.cuda()  # noqa: E731
    cache = S.PagedCache(f(c["k"]), f(c["v"]), f(c["table"]), f(c["lens"]), f(c["ks"]), f(c["vs"]))
    q = x[:, :Hq].contiguous().cuda()
    call = S.paged_append_fp8 if fp8 else S.paged_append
    k, v = x[:, Hq:Hq + Hkv].contiguous().cuda(), x[:, Hq + Hkv:].contiguous().cuda()
    k_out = torch.full_like(k, 7.0)
    call(k, v, cache, rope=c["rope"].cuda(), q=q, q_out=q, k_out=k_out)
    torch.cuda.synchronize()
    pos = np.array([n - 1 for n in c["lens"].tolist()])
    live = pos >= 0
    X = x.double().numpy()
    near16(np64(q)[live], oracle.rotate(X[live, :Hq], pos[live], c["rope"]), 8.0, BF)
    assert torch.equal(q[5].cpu(), x[5, :Hq]) and (k_out[5] == 7).all()
    if fp8:
        rk = X[:, Hq:Hq + Hkv].copy()
        rk[live] = oracle.rotate(rk[live], pos[live], c["rope"])
        want, ws = oracle.paged_append_fp8(rk, c["table"], c["lens"], c["k"], c["ks"])
        assert np.array_equal(np64(cache.k_scale), ws)
        d = oracle.fp8_e4m3_value(cache.k_pages.cpu().numpy()) - oracle.fp8_e4m3_value(want)
        assert np.count_nonzero(d) <= 2  # a code next to a tie may fall the other way
    else:
        want, wv = oracle.paged_append(np64(k_out), X[:, Hq + Hkv:], c["table"], c["lens"], c["k"], c["v"])
        assert np.array_equal(np64(cache.k_pages), want)
        assert np.array_equal(np64(cache.v_pages), wv)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_out_of_bounds_positions_write_nothing(fp8):
    """Positions past the rotation table or before 0, and pages outside the pool: the
    status is set, in-range tokens of the call are written, nothing else changes."""
    Hq, Hkv, D, page = 4, 2, 64, 16
    c = append_case([3, 4, 2, 1], [30, 0, 14, 5], Hq, Hkv, D, page, BF, 64, 43, fp8)
    c["lens"][1] = 2              # positions -2 .. 1
    c["table"][2, 1] = 10 ** 6    # a page that the call does not need
    c["table"][3, 0] = -1
    rope = c["rope"][:32]         # sequence 0 ends at position 32
    f = lambda t: None if t is None else t.cuda()  # noqa: E731
    cache = S.PagedCache(f(c["k"]), f(c["v"]), f(c["table"]), f(c["lens"]), f(c["ks"]), f(c["vs"]))
    x = c["x"][:10].cuda()
    call = S.paged_append_fp8 if fp8 else S.paged_append
    call(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, c["cu"].cuda(), rope.cuda())
    torch.cuda.synchronize()
    assert S.get_status() == 6
    S.clear_status()
    # the tokens that are in range: 0, 1 of sequence 0, 5, 6 of sequence 1, 7, 8 of sequence 2
    wrote = {(int(c["table"][0, 1]), 14), (int(c["table"][0, 1]), 15), (int(c["table"][1, 0]), 0),
             (int(c["table"][1, 0]), 1), (int(c["table"][2, 0]), 14), (int(c["table"][2, 0]), 15)}
    src = {7: (int(c["table"][2, 0]), 14), 5: (int(c["table"][1, 0]), 0)}
    for t, (at, r) in src.items():
        v = c["x"][t, Hq + Hkv:].double().numpy()
        if fp8:
            s = np64(cache.v_scale)[at][:, None]
            got = oracle.fp8_e4m3_value(cache.v_pages[at, :, r].cpu().numpy()) * s
            assert (np.abs(got - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * s)).all()
        else:
            assert np.array_equal(np64(cache.v_pages[at, :, r]), v)
    touched = {at for at, _ in wrote}
    for at in range(c["v"].shape[0]):
        for r in range(page):
            if (at, r) in wrote or (fp8 and at in touched):
                continue
            assert torch.equal(cache.v_pages[at, :, r].cpu(), c["v"][at, :, r])
            assert torch.equal(cache.k_pages[at, :, r].cpu(), c["k"][at, :, r])


@pytest.mark.parametrize("fp8", [False, True])
def test_append_offsets_past_the_tokens_write_nothing(fp8):
    """Offsets that name rows past T, or before 0: the status is set, that sequence's
    pages and scales stay as they are; the next ones are written.  So is a length
    below the sequence's new tokens, down to the type's lowest."""
    Hq, Hkv, D, page = 2, 1, 64, 16
    c = append_case([3, 20, 4, 2], [5, 9, 0, 30], Hq, Hkv, D, page, BF, None, 48, fp8)
    c["lens"][2] = -2 ** 31
    f = lambda t: None if t is None else t.cuda()  # noqa: E731
    call = S.paged_append_fp8 if fp8 else S.paged_append
    x = c["x"].cuda()
    for edit, T, bad in (([0, 3, 23, 27, 60], 29, [2, 3]), ([-1, 3, 23, 27, 29], 29, [0, 2]),
                         ([0, 3, 23, 27, 29], 10, [1, 2, 3])):
        cache = S.PagedCache(f(c["k"]), f(c["v"]), f(c["table"]), f(c["lens"]), f(c["ks"]), f(c["vs"]))
        call(x[:T, Hq:Hq + Hkv], x[:T, Hq + Hkv:], cache, torch.tensor(edit, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        assert S.get_status() == 6
        S.clear_status()
        for b in range(4):
            same = all(torch.equal(now[c["table"][b].long()].cpu(), was[c["table"][b].long()])
                       for now, was in ((cache.k_pages, c["k"]), (cache.v_pages, c["v"]),
                                        (cache.k_scale, c["ks"]), (cache.v_scale, c["vs"]))
                       if was is not None)
            assert same == (b in bad), (edit, b)


@pytest.mark.parametrize("fp8", [False, True])
def test_the_calls_two_ways_agree(fp8):
    """A call with a stream argument takes the Python path, one without the short way
    through the extension; both allocate what is not given, and give the same bits."""
    Hq, Hkv, D, page = 8, 2, 64, 32
    c = append_case([1] * 5, [0, 31, 32, 100, 7], Hq, Hkv, D, page, F16, 32, 47, fp8)
    f = lambda t: None if t is None else t.cuda()  # noqa: E731
    x = c["x"][:5].cuda()
    res = []
    for stream in (None, torch.cuda.current_stream()):
        cache = S.PagedCache(f(c["k"]), f(c["v"]), f(c["table"]), f(c["lens"]), f(c["ks"]), f(c["vs"]))
        append = S.paged_append_fp8 if fp8 else S.paged_append
        attend = S.paged_decode_fp8 if fp8 else S.paged_decode
        k_out = torch.empty(5, Hkv, D, dtype=F16, device="cuda")
        q = append(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, None, c["rope"].cuda(), True, x[:, :Hq],
                   k_out=k_out, stream=stream)
        out = attend(q, cache, None, n_sink=2, window=50, stream=stream)
        torch.cuda.synchronize()
        res.append([q, k_out, cache.k_pages, cache.v_pages, *out])
        assert S._short_way().paged_append(cache._at, int(fp8), cache._kind, cache._dev, x[:, :Hkv], x[:, :Hkv],
                                           None, None, False, x[:, :Hq], None, None) == -1
        assert S._short_way().paged_decode(cache._at, 1 - int(fp8), cache._kind, cache._dev, q, None, 0, 0,
                                           None, q, out[0], out[1], out[2]) == -1
    assert all(torch.equal(a, b) for a, b in zip(*res))
    with pytest.raises(S.SinkAttnError, match="WORKSPACE"):
        attend(q, cache, None, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(S.SinkAttnError, match="INVALID_ARG"):
        attend(q, cache, None, window=-1)


@pytest.mark.parametrize("fp8", [False, True])
def test_what_a_call_allocates_belongs_to_its_stream(fp8):
    """Results and workspace of a call with a stream argument come from that stream's
    memory: the current stream's could still be in use, or be given out again."""
    Hq, Hkv, D, page = 4, 2, 64, 16
    c = append_case([1, 1], [600, 5], Hq, Hkv, D, page, BF, None, 50, fp8)
    f = lambda t: None if t is None else t.cuda()  # noqa: E731
    cache = S.PagedCache(f(c["k"]), f(c["v"]), f(c["table"]), f(c["lens"]), f(c["ks"]), f(c["vs"]))
    x = c["x"][:2].cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    q = (S.paged_append_fp8 if fp8 else S.paged_append)(
        x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, q=x[:, :Hq], stream=side)
    out = (S.paged_decode_fp8 if fp8 else S.paged_decode)(q, cache, None, stream=side)
    side.synchronize()

    def stream_of(t):
        at = t.data_ptr()
        return [s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= at < s["address"] + s["total_size"]]

    assert stream_of(x) == [0]
    for t in (q, *out):
        assert stream_of(t) == [side.cuda_stream]
    want = oracle.paged_decode(q, cache.k_pages, cache.v_pages, c["table"], c["lens"], 0, 0, None,
                               D ** -0.5, *(None if t is None else t.cpu() for t in (cache.k_scale, cache.v_scale)))
    tol = torch.finfo(BF).eps / 2 * np.abs(want[0]) + 2.0 ** -10 * 5
    assert (np.abs(np64(out[0]) - want[0]) <= tol).all()


def test_append_many_sequences_and_no_token():
    """More sequences than a warp's first search step covers, most without a token;
    T = 0 does nothing."""
    n = torch.randint(0, 3, (2500,), generator=gen(44)).tolist()
    c = append_case(n, [i % 40 for i in range(2500)], 4, 1, 64, 16, BF, 64, 45, False)
    cache = S.PagedCache(c["k"].cuda(), c["v"].cuda(), c["table"].cuda(), c["lens"].cuda())
    x = c["x"].cuda()
    S.paged_append(x[:0, 4:5], x[:0, 5:], cache, torch.zeros(2501, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(cache.v_pages.cpu(), c["v"])
    S.paged_append(x[:, 4:5], x[:, 5:], cache, c["cu"].cuda())
    torch.cuda.synchronize()
    wk, wv = oracle.paged_append(c["x"][:, 4:5], c["x"][:, 5:], c["table"], c["lens"], c["k"], c["v"], c["cu"])
    assert np.array_equal(np64(cache.k_pages), wk) and np.array_equal(np64(cache.v_pages), wv)


@pytest.mark.parametrize("fp8", [False, True])
def test_the_largest_batch(fp8):
    """65,535 sequences, some without a token: each block of the grid meets a run of
    them.  A sequence's result does not depend on its neighbours."""
    Hkv, D, page, B, n = 1, 64, 16, 65535, 64
    g = gen(49)
    x = torch.randn(n, 2 * Hkv + 2, D, generator=g).to(BF)
    past = torch.randint(0, page, (n,), generator=g, dtype=torch.int32)
    past[:3] = torch.tensor([0, page - 1, -1])
    k, ks = make_pool(n, Hkv, page, D, None if fp8 else BF, g)
    append = S.paged_append_fp8 if fp8 else S.paged_append
    attend = S.paged_decode_fp8 if fp8 else S.paged_decode

    def run(b):
        i = torch.arange(b) % n
        f = lambda t: None if t is None else t[i].cuda()  # noqa: E731
        table = torch.arange(b, dtype=torch.int32).view(b, 1).cuda()
        cache = S.PagedCache(f(k), f(k), table, f(past + 1), f(ks), f(ks))
        xd = f(x)
        append(xd[:, 2:3], xd[:, 3:], cache)
        out = attend(xd[:, :2].contiguous(), cache, None)
        torch.cuda.synchronize()
        return [t.cpu() for t in (cache.k_pages, cache.v_pages, *out)], i

    small, _ = run(n)
    big, i = run(B)
    assert not torch.equal(small[0], k) and bool((small[2] != 0).any())
    for a, b in zip(small, big):
        assert torch.equal(a[i], b)


@pytest.mark.parametrize("fp8", [False, True])
def test_two_threads_at_once(fp8):
    """Two Python threads, each with a stream, append to their own pages of one pool and
    attend, step after step: the same bits as one after the other."""
    Hq, Hkv, D, page, steps = 8, 2, 128, 16, 40
    c = append_case([1] * 4, [300, 7, 1000, 40], Hq, Hkv, D, page, BF, None, 52, fp8)
    width = c["table"].shape[1]
    f = lambda t: None if t is None else t.clone().cuda()  # noqa: E731
    xs = torch.randn(steps, 4, Hq + 2 * Hkv, D, generator=gen(53)).to(BF).cuda()
    append = S.paged_append_fp8 if fp8 else S.paged_append
    attend = S.paged_decode_fp8 if fp8 else S.paged_decode

    def work(pools, half, got):
        rows = slice(2 * half, 2 * half + 2)
        with torch.cuda.stream(torch.cuda.Stream()):
            lens = c["lens"][rows].cuda() - steps
            lens.clamp_(min=0)
            cache = S.PagedCache(pools[0], pools[1], c["table"][rows].contiguous().cuda(), lens, *pools[2:])
            for i in range(steps):
                x = xs[i, rows]
                lens.add_(1)
                q = append(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, q=x[:, :Hq])
                got[half].append(attend(q, cache, None)[0])
            torch.cuda.current_stream().synchronize()

    res = []
    for together in (False, True):
        pools = [f(c["k"]), f(c["v"])] + ([f(c["ks"]), f(c["vs"])] if fp8 else [])
        torch.cuda.synchronize()
        got = [[], []]
        threads = [threading.Thread(target=work, args=(pools, h, got)) for h in range(2)]
        for t in threads:
            t.start()
            if not together:
                t.join()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert len(got[0]) == len(got[1]) == steps and width >= 63
        res.append([t.cpu() for t in [*got[0], *got[1], *pools]])
    assert all(torch.equal(a, b) for a, b in zip(*res))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_then_steps_as_a_server_runs_them(fp8):
    """A prefill whose rotated queries and keys go through the forward while its pages
    fill, then decode steps (append, attend) as one captured graph, against the
    oracle on the dense sequences."""
    Hq, Hkv, D, page, steps = 8, 2, 128, 16, 20
    prompt = [37, 1, 150]
    g = gen(46)
    B, T = 3, sum(prompt)
    cap = max(prompt) + steps
    table, n = make_table([cap] * B, page, g)
    pool = (torch.uint8 if fp8 else BF)
    kp = torch.zeros(n, Hkv, page, D, dtype=pool, device="cuda")
    sc = (torch.zeros(n, Hkv, device="cuda"), torch.zeros(n, Hkv, device="cuda")) if fp8 else ()
    lens = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    cache = S.PagedCache(kp, torch.zeros_like(kp), table.cuda(), lens, *sc)
    append = S.paged_append_fp8 if fp8 else S.paged_append
    attend = S.paged_decode_fp8 if fp8 else S.paged_decode
    rope = torch.from_numpy(oracle.rope_table(cap, D)).float().cuda()
    sink = torch.randn(Hq, generator=g)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(BF)
    xd = x.cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(prompt)]), dtype=torch.int32)
    k_rot = torch.empty(T, Hkv, D, dtype=BF, device="cuda")
    q_rot = append(xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], cache, cu.cuda(), rope, q=xd[:, :Hq], k_out=k_rot)
    m = S.Mask(cu.cuda(), max(prompt))
    plan = S.Plan(T, Hq, Hkv, m)
    out, lse, _ = S.fwd(q_rot, k_rot, xd[:, Hq + Hkv:].contiguous(), sink.cuda(), m, plan)
    torch.cuda.synchronize()
    ro, rl, _ = oracle.fwd(q_rot, k_rot, x[:, Hq + Hkv:], sink, D ** -0.5, causal=True, cu_seqlens=cu)
    assert np.abs(np64(out) - ro).max() <= 2e-2
    check_lse(np64(lse), rl, 1e-3)

    step_x = torch.zeros(B, Hq + 2 * Hkv, D, dtype=BF, device="cuda")
    one = torch.ones_like(lens)
    ws = torch.empty(S.paged_decode_workspace_bytes(B, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    sd = sink.cuda()

    def step():
        lens.add_(one)
        q = append(step_x[:, Hq:Hq + Hkv], step_x[:, Hq + Hkv:], cache, rope=rope, q=step_x[:, :Hq])
        return attend(q, cache, sd, workspace=ws), q

    xs = torch.randn(steps, B, Hq + 2 * Hkv, D, generator=g).to(BF)
    step_x.copy_(xs[0])
    step()
    torch.cuda.synchronize()
    lens.sub_(one)  # the capture below takes the first step again
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, q = step()
    for i in range(steps):
        step_x.copy_(xs[i])
        graph.replay()
    torch.cuda.synchronize()
    assert lens.tolist() == [p + steps for p in prompt]
    # the oracle's sequences: the 16-bit cache's rotated keys, or what the codes stand for
    ks, vs = (None, None) if not fp8 else (cache.k_scale.cpu(), cache.v_scale.cpu())
    want = oracle.paged_decode(q, cache.k_pages, cache.v_pages, table, lens.cpu(), 0, 0, sink, D ** -0.5,
                               ks, vs)
    tol = 2.0 ** -9 * np.abs(want[0]) + 2.0 ** -10 * 5
    assert (np.abs(np64(got[0]) - want[0]) <= tol).all()
    check_lse(np64(got[1]), want[1], 2.0 ** -12)
    # and the pages hold the sequences: keys rotated in 64 bits, values as given
    for b, p in enumerate(prompt):
        seq = torch.cat([x[cu[b]:cu[b + 1]], xs[:, b]]).double().numpy()
        pos = np.arange(p + steps)
        rk = oracle.rotate(seq[:, Hq:Hq + Hkv], pos, rope)
        at, row = table[b].numpy()[pos // page], pos % page
        for val, pages, s in ((rk, cache.k_pages, ks), (seq[:, Hq + Hkv:], cache.v_pages, vs)):
            held = pages.cpu()[at, :, row]
            if fp8:
                sc_ = s[at].double().numpy()[:, :, None]
                # a row may have been rounded twice, in the subnormals of a larger scale
                bound = np.maximum(2.0 ** -4 * np.abs(val), 2.0 ** -9 * sc_) + 2.0 ** -20
                assert (np.abs(oracle.fp8_e4m3_value(held.numpy()) * sc_ - val) <= bound).all()
            else:
                near16(held.double().numpy(), val, 8.0, BF)
