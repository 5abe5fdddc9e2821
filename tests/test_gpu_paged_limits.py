"""Paged cache on the GPU at the limits of its values: infinities through the rotation,
long sums, small weights, sink logits of any size, bad pages and offsets; chains of steps in
which an 8-bit block's scale grows."""
import numpy as np
import pytest
import torch

import oracle
from learnable_sink_b200 import sinkattn as S

from gpu_util import check_lse, check_status, np64
from test_gpu_paged import BF, F16, Problem, append_case, gen, make_pool, make_table

pytestmark = pytest.mark.gpu

KINDS = [(BF, False), (F16, False), (BF, True), (F16, True)]


@pytest.fixture(autouse=True)
def _status():
    S.clear_status()
    yield
    check_status()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,D", [(BF, 128), (F16, 64)])
def test_append_rotates_infinities(dtype, D, inter):
    """An infinite key element makes both elements of its pair infinite: the sums that the
    definition gives, +-448 s as codes and +-inf in k_out; NaN only where two infinities
    cancel, or one meets a sine or cosine of 0.  The other elements are as without it."""
    page, rot, n = 16, 32, 7
    g = gen(70 + D + inter)
    x = torch.randn(n, 2, D, generator=g).to(dtype)
    x[:, :, 40] = 100.0  # past the rotated elements: the block's scale is 2^-2
    clean = x.clone()
    ia, ib = (6, 7) if inter else (3, 3 + rot // 2)
    inf = float("inf")
    for t, (a, b) in enumerate([(inf, 1.0), (inf, 1.0), (1.0, inf), (-inf, 1.0), (2.0, -inf), (-inf, inf)]):
        x[t, 0, ia], x[t, 0, ib] = a, b
    rope = torch.from_numpy(oracle.rope_table(n, rot)).float()
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    table = torch.zeros(1, 1, dtype=torch.int32).cuda()
    got = []
    for src in (x, clean):
        codes = torch.zeros(1, 1, page, D, dtype=torch.uint8)
        c8 = S.PagedCache(codes.cuda(), codes.cuda(), table, lens, torch.zeros(1, 1).cuda(),
                          torch.zeros(1, 1).cuda())
        p16 = torch.zeros(1, 1, page, D, dtype=dtype)
        c16 = S.PagedCache(p16.cuda(), p16.cuda(), table, lens)
        k8, k16 = (torch.empty(n, 1, D, dtype=dtype, device="cuda") for _ in range(2))
        xd = src.cuda()
        S.paged_append_fp8(xd[:, :1], xd[:, 1:], c8, cu, rope.cuda(), inter, k_out=k8)
        S.paged_append(xd[:, :1], xd[:, 1:], c16, cu, rope.cuda(), inter, k_out=k16)
        torch.cuda.synchronize()
        assert float(c8.k_scale) == 0.25
        got.append((c8.k_pages[0, 0, :n].cpu(), k8[:, 0].cpu(), k16[:, 0].cpu()))
    at = 6 // 2 if inter else 3  # the pair's angle
    co, si = rope[:, at].double().numpy(), rope[:, rot // 2 + at].double().numpy()
    a, b = x[:, 0, ia].double().numpy(), x[:, 0, ib].double().numpy()
    with np.errstate(invalid="ignore"):
        want = np.stack([a * co - b * si, b * co + a * si])
    assert np.isnan(want).sum() == 2 and np.isinf(want).sum() == 10  # position 0's, and inf - inf
    (codes, k8, k16), (codes0, k80, k160) = got
    for i, w in zip((ia, ib), want):
        for t in range(n):
            c, o8, o16 = int(codes[t, i]), float(k8[t, i]), float(k16[t, i])
            if np.isnan(w[t]):
                assert c & 0x7F == 0x7F and np.isnan(o8) and np.isnan(o16), (t, i)
            elif np.isinf(w[t]):
                assert c == (0x7E if w[t] > 0 else 0xFE) and o8 == o16 == w[t], (t, i, c, o8, o16)
    rest = [i for i in range(D) if i not in (ia, ib)]
    for u, v in zip(got[0], got[1]):
        assert torch.equal(u[:, rest], v[:, rest]) and torch.equal(u[6], v[6])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,G", [(64, 4), (128, 4), (128, 8)])
def test_decode_sums_over_a_long_row(fp8, D, G):
    """262,144 equal weights in a row that is not cut: the result is the values' mean, rounded
    once.  The tensor cores truncate a sum as they add to it (less than 2^-23 of it for
    each step of 16 positions), over 16 tiles of 128 positions at most: 2^-16; the sums of
    those, 128 at most, and the weights' own add 2^-17."""
    n, page = 262144, 128
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    pages = n // page
    v = torch.rand(pages, 1, page, D, generator=torch.Generator("cuda").manual_seed(90), device="cuda") + 0.5
    sc = ()
    if fp8:
        v = (v * 128).to(torch.float8_e4m3fn)
        sc = (torch.full((pages, 1), 2.0 ** -7, device="cuda"),) * 2
        value = v.double() * 2.0 ** -7
    else:
        v = v.to(F16)
        value = v.double()
    table = torch.arange(pages, dtype=torch.int32).expand(B, pages).contiguous().cuda()
    cache = S.PagedCache(torch.zeros_like(v), v, table, torch.full((B,), n, dtype=torch.int32).cuda(), *sc)
    call = S.paged_decode_fp8 if fp8 else S.paged_decode
    out, lse, _ = call(torch.ones(B, G, D, dtype=F16, device="cuda"), cache, None)
    want = value.mean((0, 1, 2))
    d = (out.double() / want - 1).abs().max().item()
    assert d <= 2.0 ** -11 + 2.0 ** -16 + 2.0 ** -17, d
    check_lse(np64(lse), np.full((B, G), np.log(n)), 2.0 ** -18)


@pytest.mark.parametrize("D,n_sink,window", [(64, 0, 0), (128, 0, 0), (64, 4, 40000)])
def test_decode_lse_of_small_weights_beside_a_dominant_one(D, n_sink, window):
    """The first token's weight is 1, every other one's 2^-20.3, in rows that are not cut: a
    thread's sum begins with the large one, and the small ones must not be lost to it (16 of
    them in a row lose at most 2^-20).  The scores are off by 2^-17.7 at most."""
    n, page = 131072, 128
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    k = torch.zeros(n // page, 1, page, D, dtype=BF, device="cuda")
    k[0, 0, 0, 0] = 14.0
    table = torch.arange(n // page, dtype=torch.int32).expand(B, n // page).contiguous().cuda()
    cache = S.PagedCache(k, torch.zeros_like(k), table, torch.full((B,), n, dtype=torch.int32).cuda())
    q = torch.zeros(B, 4, D, dtype=BF, device="cuda")
    q[:, :, 0] = 8.0
    lse = S.paged_decode(q, cache, None, n_sink=n_sink, window=window,
                         scale=20.3 * float(np.log(2.0)) / 112.0)[1]
    seen = n if window == 0 else window + n_sink
    check_lse(np64(lse), np.full((B, 4), 20.3 * np.log(2.0) + np.log1p((seen - 1) * 2.0 ** -20.3)), 2.0 ** -16)


@pytest.mark.parametrize("dtype,fp8", KINDS)
@pytest.mark.parametrize("D,n_sink,window", [(64, 0, 0), (128, 0, 0), (64, 4, 40000)])
@pytest.mark.parametrize("below,lift", [(20.3, 0), (23.7, 0), (25.5, 0), (27.5, 0), (20.3, 5)])
def test_decode_small_weights_beside_a_dominant_one(dtype, fp8, D, n_sink, window, below, lift):
    """The first token takes nearly all of the weight, every other one 2^-below of it, and
    all share one reference: one or two equal sequences for each block that fits the GPU, so
    that none is cut.  Values are 0 in the first token's page and 1 elsewhere, so the output is the
    small weights' sum.  A weight is off by at most 2^-16 of itself and 2^-30 of the largest
    (the latter times 2^lift, the first page's value scale over the others'); the result is
    rounded once more; the sums of 16 tiles (2^-16), their own and the scores' errors add less
    than 2^-12 of it."""
    n, page = 131072, 128
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    pages = n // page
    k = torch.zeros(pages, 1, page, D, device="cuda")
    v = torch.ones(pages, 1, page, D, device="cuda")
    k[0, 0, 0, 0] = 14.0
    v[0] = 0
    sc = ()
    if fp8:
        k, v = (t.to(torch.float8_e4m3fn) for t in (k, v))
        sc = (torch.ones(pages, 1, device="cuda"), torch.ones(pages, 1, device="cuda"))
        sc[1][0] = 2.0 ** lift
    else:
        k, v = k.to(dtype), v.to(dtype)
    table = torch.arange(pages, dtype=torch.int32).expand(B, pages).contiguous()
    cache = S.PagedCache(k, v, table.cuda(), torch.full((B,), n, dtype=torch.int32).cuda(), *sc)
    q = torch.zeros(B, 4, D, dtype=dtype)
    q[:, :, 0] = 8.0
    call = S.paged_decode_fp8 if fp8 else S.paged_decode
    out, lse, ss = call(q.cuda(), cache, None, n_sink=n_sink, window=window,
                        scale=below * float(np.log(2.0)) / 112.0)
    torch.cuda.synchronize()
    seen = n if window == 0 else window + n_sink
    held = n - page if window == 0 else window  # those of value 1
    w = 2.0 ** -below
    want = held * w / (1 + (seen - 1) * w)
    tol = want * (torch.finfo(dtype).eps / 2 + 2.0 ** -16 + 2.0 ** -12) + \
        held * 2.0 ** -30 * (2.0 ** lift if fp8 else 1)
    d = np.abs(np64(out) - want).max()
    assert d <= tol, (d / want, tol / want)
    # the score's float32 product is off by 2^-23 of `below` log2 units or so
    check_lse(np64(lse), np.full((B, 4), below * np.log(2.0) + np.log1p((seen - 1) * w)), 2.0 ** -16)
    assert np.abs(np64(ss) - 1).max() <= 2.0 ** -20


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_sink_logits_of_any_size(fp8):
    """A sink logit so large that the keys have no weight left, +inf among them, takes all of
    it: out = 0, the gate 0, lse = a_h.  One so low that it has none is as no sink, and is
    still lse where a sequence sees no key.  Whole sequences and split ones."""
    top = float(torch.finfo(torch.float32).max)
    a = [float("inf"), top, 3.0e38, 1e30, -top, -2.2e38, -1e30, -float("inf")]
    p = Problem([9000, 100, 0], 8, 2, 128, 32, BF, fp8, seed=81)
    p.sink = None
    none = p.want()
    p.sink = torch.tensor(a)
    out, lse, ss = (t.cpu() for t in p.run())
    sink = p.sink.expand(3, 8)
    assert (out[:, :4] == 0).all() and (ss[:, :4] == 0).all()
    assert torch.equal(lse[:, :4], sink[:, :4])
    assert torch.equal(lse[2], sink[2]) and (out[2] == 0).all() and (ss[2] == 0).all()
    p.check([t[:2, 4:] for t in (out, lse, ss)], [w[:2, 4:] for w in none])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("single", [False, True])
def test_append_with_a_bad_page_still_rotates_the_queries(fp8, single):
    """A token whose page is outside the pool, or past the table, writes no key and no value,
    nor k_out, and sets the status; its query, which needs the position alone, is rotated.
    One without a valid position leaves all of its outputs as they were."""
    Hq, Hkv, D, page = 4, 2, 64, 16
    new = [1] * 5 if single else [2, 3, 1, 2, 1]
    c = append_case(new, [20, 16, 3, 40, 70], Hq, Hkv, D, page, BF, 64, 80, fp8)
    width = c["table"].shape[1]
    c["table"][0, 1] = -1
    c["table"][1, 1] = c["k"].shape[0]
    c["lens"][3] = width * page + 1 if single else width * page + 2  # every new position is past the table
    rope = torch.from_numpy(oracle.rope_table(width * page + 2, 64)).float()
    c["lens"][4] = -7 if not single else width * page + 40  # below the new tokens; past the rotation table
    T = sum(new)
    x = c["x"][:T].cuda()
    f = lambda t: None if t is None else t.cuda()  # noqa: E731
    cache = S.PagedCache(f(c["k"]), f(c["v"]), f(c["table"]), f(c["lens"]), f(c["ks"]), f(c["vs"]))
    q_out = torch.full((T, Hq, D), 7.0, dtype=BF, device="cuda")
    k_out = torch.full((T, Hkv, D), 7.0, dtype=BF, device="cuda")
    (S.paged_append_fp8 if fp8 else S.paged_append)(
        x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, None if single else c["cu"].cuda(), rope.cuda(),
        q=x[:, :Hq], q_out=q_out, k_out=k_out)
    torch.cuda.synchronize()
    assert S.get_status() == 6
    S.clear_status()
    X = c["x"][:T].double().numpy()
    cu, lens = c["cu"].tolist(), c["lens"].tolist()
    touched = torch.zeros(c["k"].shape[0], dtype=torch.bool)
    for b in range(5):
        for t in range(cu[b], cu[b + 1]):
            pos = lens[b] - (cu[b + 1] - t)
            if b == 4:
                assert (q_out[t] == 7).all() and (k_out[t] == 7).all()
                continue
            want = oracle.rotate(X[t:t + 1, :Hq], [pos], rope)[0]
            assert (np.abs(np64(q_out[t]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18).all(), (b, t)
            assert bool((k_out[t] == 7).all()) == (b != 2), (b, t)
            if b == 2:
                touched[c["table"][2, pos // page].long()] = True
    for now, was in ((cache.k_pages, c["k"]), (cache.v_pages, c["v"]), (cache.k_scale, c["ks"]),
                     (cache.v_scale, c["vs"])):
        if was is not None:
            assert torch.equal(now.cpu()[~touched], was[~touched])
    assert not torch.equal(cache.v_pages.cpu()[touched], c["v"][touched])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("offsets,bad", [([0, 3, 5, 9], [2]), ([0, 5, 5, 6], [2]), ([-4, -1, 2, 5], [0, 1]),
                                         ([0, 2, 4, 2 ** 31 - 1], [2])])
def test_append_offsets_wholly_outside_set_the_status(fp8, offsets, bad):
    """Offsets that reach past T or below 0 set the status even where no row of the call is
    theirs; the sequences inside are written."""
    c = append_case([2, 2, 1], [8, 10, 25], 2, 1, 64, 16, BF, None, 82, fp8)
    f = lambda t: None if t is None else t.cuda()  # noqa: E731
    cache = S.PagedCache(f(c["k"]), f(c["v"]), f(c["table"]), f(c["lens"]), f(c["ks"]), f(c["vs"]))
    x = c["x"][:5].cuda()
    (S.paged_append_fp8 if fp8 else S.paged_append)(
        x[:, 2:3], x[:, 3:], cache, torch.tensor(offsets, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert S.get_status() == 6
    S.clear_status()
    for b in range(3):
        rows = c["table"][b].long()
        same = torch.equal(cache.v_pages.cpu()[rows], c["v"][rows])
        n = offsets[b + 1] - offsets[b]
        assert same == (b in bad or n == 0), b


@pytest.mark.parametrize("D,page", [(64, 16), (128, 32)])
def test_steps_whose_scales_grow(D, page):
    """Append and attend step after step without a wait, values half as large again each
    step, so that blocks are re-encoded to a larger scale under the kernel before: each
    step's result belongs to that step's codes and scales."""
    Hq, Hkv, steps = 16, 8, 24
    past = [0, page - 3, 200]
    g = gen(83)
    table, n = make_table([p + steps for p in past], page, g)
    k, ks = make_pool(n, Hkv, page, D, None, g)
    v, vs = make_pool(n, Hkv, page, D, None, g)
    lens = torch.tensor(past, dtype=torch.int32)
    xs = torch.randn(steps, 3, Hq + 2 * Hkv, D, generator=g)
    xs[:, :, Hq:] *= 1.5 ** torch.arange(steps).float()[:, None, None, None] * 0.01
    xs = xs.to(BF)
    sink = torch.randn(Hq, generator=g)
    cache = S.PagedCache(k.cuda(), v.cuda(), table.cuda(), lens.cuda(), ks.cuda(), vs.cuda())
    xd, sd, one = xs.cuda(), sink.cuda(), torch.ones(3, dtype=torch.int32, device="cuda")
    ws = torch.empty(S.paged_decode_workspace_bytes(3, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    qs = xd[:, :, :Hq].contiguous()
    torch.cuda.synchronize()
    got = []
    for i in range(steps):
        cache.cache_seqlens.add_(one)
        S.paged_append_fp8(xd[i, :, Hq:Hq + Hkv], xd[i, :, Hq + Hkv:], cache)
        got.append(S.paged_decode_fp8(qs[i], cache, sd, workspace=ws))
    torch.cuda.synchronize()
    kc, vc, ksn, vsn = k.numpy(), v.numpy(), ks.double().numpy(), vs.double().numpy()
    grown = 0
    for i in range(steps):
        lens = lens + 1
        was = vsn
        kc, ksn = oracle.paged_append_fp8(xs[i, :, Hq:Hq + Hkv], table, lens, kc, ksn)
        vc, vsn = oracle.paged_append_fp8(xs[i, :, Hq + Hkv:], table, lens, vc, vsn)
        grown += int((vsn > was).sum())
        want = oracle.paged_decode(xs[i, :, :Hq], kc, vc, table, lens, 0, 0, sink, D ** -0.5, ksn, vsn)
        top = (np.abs(oracle.fp8_e4m3_value(vc)) * vsn[:, :, None, None])[table.numpy()].max()
        kmax = (np.abs(oracle.fp8_e4m3_value(kc)) * ksn[:, :, None, None])[table.numpy()].max()
        qsum = xs[i, :, :Hq].abs().double().sum(-1).max().item()
        # the error of a score's D float32 products, and a weight's, twice that
        err = (D + 3) * 2.0 ** -24 * qsum * kmax * D ** -0.5
        d = np.abs(np64(got[i][0]) - want[0])
        assert (d <= 2.0 ** -8 * np.abs(want[0]) + (2.0 ** -10 + 2 * err) * top).all(), i
        check_lse(np64(got[i][1]), want[1], 2.0 ** -12 + err)
    assert grown > 100
    assert np.array_equal(cache.k_pages.cpu().numpy(), kc) and np.array_equal(np64(cache.k_scale), ksn)
    assert np.array_equal(cache.v_pages.cpu().numpy(), vc) and np.array_equal(np64(cache.v_scale), vsn)


@pytest.mark.parametrize("dtype,fp8", KINDS)
@pytest.mark.parametrize("D,G", [(64, 8), (128, 4), (64, 16), (128, 16)])
def test_decode_folded_sums_follow_the_references(dtype, fp8, D, G):
    """Scores that rise twice, by 7 log2 units in all, behind the first folds of a row that is not
    cut, and fall again: what was folded is brought along each time."""
    n, page = 45000, 64
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    p = Problem([n], G, 1, D, page, dtype, fp8, seed=91)
    pages = p.table[0].long()
    pos = torch.arange(pages.numel() * page).view(-1, page)
    lift = (pos > 9000) * 2.0 + (pos > 20000) * 3.0 - (pos > 36000) * 6.0  # score units
    p.q[:, :, 0] = 8.0
    x = lift / (8.0 * p.scale)
    if fp8:
        keys = torch.randn(p.k.shape, generator=gen(92))
        keys[pages, 0, :, 0] = x
        p.ks[:] = 2.0 ** -5
        p.k = (keys * 32).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        p.k[pages, 0, :, 0] = x.to(dtype)
    want = p.want()
    p.table, p.lens = p.table.expand(B, -1).contiguous(), p.lens.expand(B).contiguous()
    p.q = p.q.expand(B, -1, -1).contiguous()
    out, lse, ss = p.run()
    assert all(torch.equal(t, t[:1].expand_as(t)) for t in (out, lse, ss))
    top = np.abs((oracle.fp8_e4m3_value(p.v.numpy()) * p.vs.double().numpy()[:, :, None, None]) if fp8
                 else np64(p.v)).max()
    d = np.abs(np64(out[0]) - want[0][0])
    tol = torch.finfo(dtype).eps / 2 * np.abs(want[0][0]) + 2.0 ** -12 * top
    assert (d <= tol).all(), float((d / tol).max())
    check_lse(np64(lse[0]), want[1][0], 2.0 ** -12)
    assert np.abs(np64(ss[0]) - want[2][0]).max() <= 2.0 ** -12


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_values_at_the_end_of_the_range(fp8):
    """Values of 1e38 and 3e38: a weight does not push their sums out of float32's range while
    the sum of e^(x - m) v is inside."""
    page = 16
    g = gen(93)
    lens = torch.tensor([1, 2, 1, 40], dtype=torch.int32)
    table = torch.arange(4 * 3, dtype=torch.int32).view(4, 3)
    k = torch.randn(12, 2, page, 128, generator=g)
    v = torch.randn(12, 2, page, 128, generator=g).sign() * torch.tensor([3e38, 1e38, 1.5e38, 4e36]
                                                                         ).repeat_interleave(3)[:, None, None, None]
    q = torch.randn(4, 8, 128, generator=g).to(BF)
    sc = ()
    if fp8:
        sc = (torch.full((12, 2), 2.0 ** -6), torch.full((12, 2), 2.0 ** 120))
        k, v = (k * 64).to(torch.float8_e4m3fn), (v / 2.0 ** 120).to(torch.float8_e4m3fn)
    else:
        k, v = k.to(BF), v.to(BF)
    cache = S.PagedCache(k.cuda(), v.cuda(), table.cuda(), lens.cuda(), *(t.cuda() for t in sc))
    out, lse, _ = (S.paged_decode_fp8 if fp8 else S.paged_decode)(q.cuda(), cache, None)
    codes = (t.view(torch.uint8) if fp8 else t for t in (k, v))
    want = oracle.paged_decode(q, *codes, table, lens, 0, 0, None, 128 ** -0.5, *sc)
    top = np.abs(want[0]).max(axis=(1, 2), keepdims=True)
    d = np.abs(np64(out) - want[0])
    assert (d <= 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -10 * top).all(), (np64(out)[:, 0, 0], want[0][:, 0, 0])
    check_lse(np64(lse), want[1], 2.0 ** -12)


@pytest.mark.parametrize("bits", [0x7FC00000, 0x7FFFFFFF, -1])
def test_decode_value_scale_that_is_not_a_number(bits):
    """A value scale of NaN or below 0 is outside the contract; it makes the page's head NaN and does
    not hide its rows."""
    p = Problem([100, 100], 8, 2, 64, 16, BF, True, seed=94)
    want = p.want()
    p.vs.view(torch.int32)[p.table[0, 3].long(), 1] = bits
    p.vs[p.table[1, 2].long(), 0] = -1.0
    out, lse, ss = p.run()
    assert torch.isnan(out[0, 4:]).all() and torch.isnan(out[1, :4]).all()
    assert torch.isfinite(out[0, :4]).all() and torch.isfinite(out[1, 4:]).all()
    check_lse(np64(lse), want[1], 2.0 ** -12)
    assert np.abs(np64(ss) - want[2]).max() <= 2.0 ** -12


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_append_rotation_that_overflows(inter, sign):
    """A rotation table with a factor of its own, and keys near the end of bf16's range: a product
    beyond float32 is infinite with its sign, and saturates; it is not NaN."""
    rot, D = 16, 64
    rope = torch.tensor([[0.5] * 8 + [1.5 * sign] * 8])
    x = torch.zeros(1, 2, D, dtype=BF)
    x[:, 0, :rot] = 3.3e38
    x[:, :, 40] = 100.0
    one = torch.ones(1, dtype=torch.int32).cuda()
    codes = torch.zeros(1, 1, 16, D, dtype=torch.uint8).cuda()
    cache = S.PagedCache(codes, codes.clone(), torch.zeros(1, 1, dtype=torch.int32).cuda(), one,
                         torch.zeros(1, 1).cuda(), torch.zeros(1, 1).cuda())
    k_out = torch.empty(1, 1, D, dtype=BF, device="cuda")
    xd = x.cuda()
    S.paged_append_fp8(xd[:, :1], xd[:, 1:], cache, None, rope.cuda(), inter, k_out=k_out)
    torch.cuda.synchronize()
    # a' = 0.5 a - 1.5 sign b, b' = 0.5 b + 1.5 sign a: the second product is +-infinite
    a = torch.arange(0, rot, 2) if inter else torch.arange(rot // 2)
    b = a + 1 if inter else a + rot // 2
    up, down = (0x7E, 0xFE) if sign > 0 else (0xFE, 0x7E)
    assert float(cache.k_scale) == 0.25
    assert (codes[0, 0, 0, a.cuda()] == down).all() and (codes[0, 0, 0, b.cuda()] == up).all()
    assert (k_out[0, 0, a.cuda()] == -sign * float("inf")).all() and (k_out[0, 0, b.cuda()] == sign * float("inf")).all()
