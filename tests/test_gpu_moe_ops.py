"""Routing, slot order, combination and their backward passes on the GPU
against plain 64-bit forms."""

import numpy as np
import pytest
import torch

import ops_helpers as H
from ops_helpers import B, DT, Guarded, f64, ptr, stream, strided

pytestmark = pytest.mark.gpu


def logits_for(T, E, dtype, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * spread).to(DT[dtype]).cuda()


def run_route(x, c, bias=None, mask=None, dtype="f32", stride=None, shift=0):
    T, E = x.shape
    xs = strided(x, stride or E, shift)
    r = B.Router(dtype, E, c["k"], score=c["score"], n_groups=c.get("groups", 1), top_groups=c.get("top_groups", 1),
                 group_top=c.get("group_top", 1), renormalise=c["renorm"], scale=c.get("scale", 1.0))
    ids, w = Guarded(T, c["k"], torch.int32), Guarded(T, c["k"], torch.float32)
    B.reshard_moe_route(r, T, xs.ptr, xs.stride, ptr(bias), ptr(mask), ids.ptr, w.ptr, stream())
    torch.cuda.synchronize()
    assert ids.intact() and w.intact() and xs.intact()
    return ids.t, w.t


def check_route(x, c, bias=None, mask=None, **kw):
    ids, w = run_route(x, c, bias, mask, **kw)
    want, ww, tol = H.route(f64(x), c, None if bias is None else f64(bias), None if mask is None else mask.cpu().numpy())
    assert np.array_equal(ids.cpu().numpy(), want)
    H.close(f64(w), ww, np.abs(ww) * tol[:, None], "f32", "weights")


ROUTERS = [
    (1, 256, dict(k=8, score="sigmoid", renorm=True, groups=8, top_groups=4, group_top=2, scale=2.5), True),
    (33, 256, dict(k=8, score="sigmoid", renorm=True, groups=8, top_groups=4, group_top=2, scale=2.5), True),
    (50, 128, dict(k=8, score="softmax", renorm=True), False),
    (50, 128, dict(k=8, score="softmax", renorm=False), True),
    (17, 160, dict(k=6, score="softmax", renorm=False, groups=8, top_groups=3, scale=16.0), False),
    (17, 160, dict(k=6, score="softmax", renorm=True, groups=8, top_groups=3, group_top=2), False),
    (19, 60, dict(k=4, score="softmax", renorm=True), False),
    (19, 60, dict(k=4, score="sigmoid", renorm=False, groups=3, top_groups=2, group_top=2), True),
    (21, 60, dict(k=3, score="sigmoid", renorm=True, groups=12, top_groups=5, group_top=2), True),
    (5, 1, dict(k=1, score="softmax", renorm=True), True),
    (5, 8, dict(k=8, score="sigmoid", renorm=True), False),
    (5, 32, dict(k=32, score="softmax", renorm=True), True),
    (9, 1024, dict(k=32, score="sigmoid", renorm=True, groups=16, top_groups=16, group_top=1), True),
    (9, 1000, dict(k=17, score="softmax", renorm=False), False),
    (40, 16, dict(k=2, score="softmax", renorm=True, groups=16, top_groups=2, group_top=2), False),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", range(len(ROUTERS)))
def test_route(case, dtype):
    T, E, c, biased = ROUTERS[case]
    x = logits_for(T, E, dtype, 10 + case)
    bias = (torch.randn(E, generator=torch.Generator().manual_seed(5)) * 0.05).cuda() if biased else None
    check_route(x, c, bias, dtype=dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_strides_and_misaligned_rows(dtype):
    x = logits_for(37, 96, dtype, 3)
    check_route(x, dict(k=4, score="softmax", renorm=True), dtype=dtype, stride=101, shift=3)


def test_route_equal_scores_go_to_the_lowest_expert():
    x = torch.zeros(7, 64, device="cuda")
    x[1, 40:] = 1.0
    x[2, ::2] = 1.0
    for c in (dict(k=8, score="softmax", renorm=True), dict(k=8, score="sigmoid", renorm=True),
              dict(k=4, score="sigmoid", renorm=True, groups=8, top_groups=2, group_top=2)):
        check_route(x, c)
        check_route(x, c, bias=torch.full((64,), 0.25, device="cuda"))
    check_route(x.bfloat16(), dict(k=8, score="softmax", renorm=True), dtype="bf16")


def test_route_tells_scores_apart_that_float32_does_not():
    """Sigmoid scores near 1 with a bias: pairs whose float32 scores are equal
    or reversed by rounding, in both orders."""
    rng = np.random.default_rng(0)
    x = torch.tensor(rng.normal(0, 1, (400, 64)), dtype=torch.float32)
    x[:, 1::2] = torch.nextafter(x[:, ::2], torch.full_like(x[:, ::2], 9.0))   # one float32 step higher
    x[::2] = x[::2].flip(1)
    bias = torch.zeros(64)
    for b in (None, bias, bias + 0.4):
        check_route(x.cuda(), dict(k=8, score="sigmoid", renorm=True), None if b is None else b.cuda())
        check_route(x.cuda() * 4 + 9, dict(k=8, score="sigmoid", renorm=True), None if b is None else b.cuda())
        check_route(x.cuda(), dict(k=8, score="softmax", renorm=False, groups=4, top_groups=2, group_top=2),
                    None if b is None else b.cuda())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_masked_logits(score, groups):
    """-infinity and NaN logits, the type's lowest value, whole rows without a
    candidate, fewer candidates than slots, padding tokens."""
    x = logits_for(24, 32, "f32", 8)
    x[1] = -float("inf")
    x[2] = float("nan")
    x[3, 3:] = -float("inf")
    x[4, :30] = float("nan")
    x[5] = torch.finfo(torch.float32).min
    x[6, 5:] = torch.finfo(torch.float32).min
    x[7, ::3] = -float("inf")
    x[8, 4] = 80.0
    x[9, 9] = -200.0
    mask = torch.ones(24, dtype=torch.uint8, device="cuda")
    mask[12:15] = 0
    mask[16] = 7
    for renorm in (True, False):
        c = dict(k=4, score=score, renorm=renorm, groups=groups, top_groups=min(groups, 2), group_top=2 if groups > 1 else 1)
        check_route(x, c, mask=mask)
        check_route(x, c, bias=torch.linspace(-0.1, 0.1, 32, device="cuda"), mask=mask)


def test_route_infinite_logits():
    x = logits_for(4, 32, "f32", 8)
    x[1, 7] = float("inf")
    x[2, 7] = x[2, 9] = float("inf")
    for score in ("softmax", "sigmoid"):
        check_route(x, dict(k=3, score=score, renorm=True))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (35, 128, 8), (17, 60, 4), (6, 1000, 32), (5, 1, 1), (9, 16, 17)])
def test_route_grad(dtype, score, renorm, T, E, k):
    x = logits_for(T, E, dtype, T + E)
    rng = np.random.default_rng(k)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)   # some experts twice
    if T > 4:
        ids[1, :] = -1
        ids[2, 0] = -1
        ids[3, 0] = E
        ids[4, :] = ids[4, 0]
    dw = rng.normal(0, 1, (T, k)).astype(np.float32)
    c = dict(score=score, renorm=renorm, scale=2.5)
    r = B.Router(dtype, E, min(k, E), score=score, renormalise=renorm, scale=2.5)
    r.top_k = k if k <= E else min(k, E)
    ids, dw = np.ascontiguousarray(ids[:, :r.top_k]), np.ascontiguousarray(dw[:, :r.top_k])
    xs = strided(x, E + 5, 1)
    out = Guarded(T, E, DT[dtype], E + 3, 1)
    B.reshard_moe_route_grad(r, T, xs.ptr, xs.stride, ptr(torch.from_numpy(ids).cuda()),
                             ptr(torch.from_numpy(dw).cuda()), out.ptr, out.stride, stream())
    torch.cuda.synchronize()
    want, tol = H.route_grad(f64(x), ids, dw.astype(np.float64), c)
    H.close(f64(out.t), want, tol, dtype, "dlogits")
    assert out.intact()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_grad_masked_logits(score):
    x = logits_for(5, 32, "f32", 1)
    x[0, 3] = -float("inf")
    x[1, 4] = float("nan")
    x[2] = -float("inf")
    x[3, 5:] = torch.finfo(torch.float32).min
    ids = np.array([[3, 1], [4, 2], [0, 1], [9, 2], [1, 1]], dtype=np.int32)
    dw = np.ones((5, 2), dtype=np.float32)
    for renorm in (True, False):
        out = torch.full((5, 32), 7.0, device="cuda")
        r = B.Router("f32", 32, 2, score=score, renormalise=renorm)
        B.reshard_moe_route_grad(r, 5, ptr(x), 32, ptr(torch.from_numpy(ids).cuda()), ptr(torch.from_numpy(dw).cuda()),
                                 ptr(out), 32, stream())
        want, tol = H.route_grad(f64(x), ids, dw.astype(np.float64), dict(score=score, renorm=renorm))
        H.close(f64(out), want, tol, "f32", "dlogits")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_against_differences(score, renorm):
    """Central differences of the forward reference in 64 bits (step 1e-5:
    their own error is near 1e-10), against the kernel's float32 gradient."""
    x = logits_for(3, 16, "f32", 4)
    r = B.Router("f32", 16, 4, score=score, renormalise=renorm, scale=1.5)
    ids, w = torch.empty(3, 4, dtype=torch.int32, device="cuda"), torch.empty(3, 4, device="cuda")
    B.reshard_moe_route(r, 3, ptr(x), 16, None, None, ptr(ids), ptr(w), stream())
    g = torch.randn(3, 4, generator=torch.Generator().manual_seed(2)).cuda()
    out = torch.empty(3, 16, device="cuda")
    B.reshard_moe_route_grad(r, 3, ptr(x), 16, ptr(ids), ptr(g), ptr(out), 16, stream())
    i, base, gg = ids.cpu().numpy(), f64(x), f64(g)

    def loss(v):
        s, _ = H.scores(v, score)
        p = np.take_along_axis(s, i, 1)
        return (1.5 * gg * (p / p.sum(1, keepdims=True) if renorm else p)).sum(1)

    _, tol = H.route_grad(base, i, gg, dict(score=score, renorm=renorm, scale=1.5))
    for e in range(16):
        hi, lo = base.copy(), base.copy()
        hi[:, e] += 1e-5
        lo[:, e] -= 1e-5
        H.close(f64(out)[:, e], (loss(hi) - loss(lo)) / 2e-5, tol[:, e] + 1e-9, "f32", "column %d" % e)


@pytest.mark.parametrize("T,k,E,first,local", [
    (1, 1, 1, 0, 1), (1, 8, 256, 0, 256), (64, 8, 256, 96, 32), (700, 6, 60, 0, 60), (511, 8, 64, 0, 64),
    (512, 8, 64, 7, 50), (513, 8, 64, 0, 64), (3000, 4, 1024, 0, 1024), (5000, 2, 9, 8, 1), (40, 32, 300, 299, 1),
    (1300, 7, 5, 0, 5)])
def test_sort(T, k, E, first, local):
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, E + 3, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < 0.02] = np.iinfo(np.int32).min
    ids[rng.random((T, k)) < 0.02] = np.iinfo(np.int32).max
    need = B.reshard_moe_sort_workspace(T, k, local)
    off, tok, pos = Guarded(1, local + 1, torch.int32), Guarded(1, T * k, torch.int32), Guarded(T, k, torch.int32)
    ws = Guarded(1, need // 4, torch.int32)
    dev = torch.from_numpy(ids).cuda()
    B.reshard_moe_sort(ptr(dev), T, k, first, local, off.ptr, tok.ptr, pos.ptr, ws.ptr, need, stream())
    torch.cuda.synchronize()
    o, t, p = H.sort(ids, first, local)
    assert np.array_equal(off.t[0].cpu().numpy(), o)
    assert np.array_equal(tok.t[0].cpu().numpy(), t)
    assert np.array_equal(pos.t.cpu().numpy(), p)
    assert off.intact() and tok.intact() and pos.intact() and ws.intact()


# So many chunks of 2048 slots that running totals stand between counts and
# places: 162 over 250 experts, 600 over few.
@pytest.mark.parametrize("T,k,E,first,local", [(33100, 10, 256, 5, 250), (307000, 4, 20, 3, 9), (1048580, 1, 3, 0, 1)])
def test_sort_long(T, k, E, first, local):
    test_sort(T, k, E, first, local)


@pytest.mark.parametrize("fill", [-1, 0, 3])
def test_sort_one_expert_takes_all_or_nothing(fill):
    T, k, local = 2000, 5, 4
    ids = np.full((T, k), fill, dtype=np.int32)
    need = B.reshard_moe_sort_workspace(T, k, local)
    off = torch.empty(local + 1, dtype=torch.int32, device="cuda")
    tok, pos = torch.empty(T * k, dtype=torch.int32, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    B.reshard_moe_sort(ptr(torch.from_numpy(ids).cuda()), T, k, 0, local, ptr(off), ptr(tok), ptr(pos), ptr(ws), need, stream())
    for got, want in zip((off, tok, pos), H.sort(ids, 0, local)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_no_tokens():
    off = torch.full((5,), 9, dtype=torch.int32, device="cuda")
    B.reshard_moe_sort(None, 0, 2, 0, 4, ptr(off), None, None, None, 0, stream())
    assert off.tolist() == [0] * 5
    B.reshard_moe_route(B.Router("f32", 8, 2), 0, None, 8, None, None, None, None, stream())
    B.reshard_moe_route_grad(B.Router("f32", 8, 2), 0, None, 8, None, None, None, 8, stream())
    B.reshard_moe_combine(B.MoeCombine("bf16", "bf16", 0, 2, 8, 4), None, None, None, None, stream())
    B.reshard_moe_combine_grad(B.MoeCombine("bf16", "bf16", 0, 2, 8, 4), None, None, None, None, None, None, stream())
    # tokens but no rows: zeros
    out = torch.full((3, 8), 5.0, device="cuda")
    pos = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    B.reshard_moe_combine(B.MoeCombine("bf16", "f32", 3, 2, 8, 0), None, ptr(pos), None, ptr(out), stream())
    assert (out == 0).all()


def slots_for(T, k, rows, seed):
    """Distinct rows for most slots, -1, too large and far negative positions for the others."""
    rng = np.random.default_rng(seed)
    pos = np.full(T * k, -1, dtype=np.int32)
    n = min(rows, T * k)
    pos[rng.permutation(T * k)[:n]] = rng.permutation(rows)[:n]
    free = np.nonzero(pos < 0)[0]
    pos[free[::3]] = rows
    pos[free[1::3]] = -2 ** 31
    return pos.reshape(T, k)


COMBINES = [(1, 1, 1, 1), (1, 8, 7168, 8), (5, 8, 100, 33), (37, 6, 513, 180), (9, 2, 2056, 18), (300, 8, 64, 1200),
            (3, 32, 4099, 90), (2, 4, 40000, 7)]


@pytest.mark.parametrize("ydt,odt", [("bf16", "bf16"), ("f32", "f32"), ("f16", "bf16"), ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("T,k,Hd,rows", COMBINES)
def test_combine(ydt, odt, T, k, Hd, rows):
    g = torch.Generator().manual_seed(T * k)
    y = torch.randn(rows, Hd, generator=g).to(DT[ydt]).cuda()
    w = torch.randn(T, k, generator=g).cuda()
    pos = slots_for(T, k, rows, Hd)
    dev = torch.from_numpy(pos).cuda()
    for pad, weights in ((0, w), (16, w), (3, None)):
        ys, out = strided(y, Hd + pad, pad), Guarded(T, Hd, DT[odt], Hd + pad, pad)
        B.reshard_moe_combine(B.MoeCombine(ydt, odt, T, k, Hd, rows, Hd + pad, Hd + pad), ys.ptr, ptr(dev),
                              ptr(weights), out.ptr, stream())
        want, tol = H.combine(f64(y), pos, np.ones((T, k)) if weights is None else f64(w))
        H.close(f64(out.t), want, tol, odt, "out")
        assert out.intact()


@pytest.mark.parametrize("ydt,odt", [("bf16", "bf16"), ("f32", "f32"), ("f16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,k,Hd,rows", COMBINES)
def test_combine_grad(ydt, odt, T, k, Hd, rows):
    g = torch.Generator().manual_seed(T * k + 1)
    y = torch.randn(rows, Hd, generator=g).to(DT[ydt]).cuda()
    d = torch.randn(T, Hd, generator=g).to(DT[odt]).cuda()
    w = torch.randn(T, k, generator=g).cuda()
    pos = slots_for(T, k, rows, Hd)
    dev = torch.from_numpy(pos).cuda()
    ok = (pos >= 0) & (pos < rows)
    named = np.zeros(rows, dtype=bool)
    named[pos[ok]] = True
    for pad, weights, parts in ((0, w, "both"), (8, w, "both"), (3, None, "both"), (0, w, "dy"), (0, w, "dw")):
        ys, ds = strided(y, Hd + pad, pad), strided(d, Hd + pad, pad)
        dy, dw = Guarded(rows, Hd, DT[ydt], Hd + pad, pad), Guarded(T, k, torch.float32)
        before = dy.t.clone()
        B.reshard_moe_combine_grad(B.MoeCombine(ydt, odt, T, k, Hd, rows, Hd + pad, Hd + pad), ds.ptr,
                                   ys.ptr if parts != "dy" else None, ptr(dev), ptr(weights),
                                   dy.ptr if parts != "dw" else None, dw.ptr if parts != "dy" else None, stream())
        torch.cuda.synchronize()
        ww = np.ones((T, k)) if weights is None else f64(w)
        if parts != "dw":
            got, want = f64(dy.t), np.zeros((rows, Hd))
            for t, j in zip(*np.nonzero(ok)):
                want[pos[t, j]] = ww[t, j] * f64(d[t])
            H.close(got[named], want[named], np.abs(want[named]) * U32, ydt, "dy")
            still = torch.from_numpy(~named)
            assert torch.equal(dy.t.cpu()[still].view(-1).contiguous().view(torch.uint8),
                               before.cpu()[still].view(-1).contiguous().view(torch.uint8))
        if parts != "dy":
            want, tol = np.zeros((T, k)), np.zeros((T, k))
            for t, j in zip(*np.nonzero(ok)):
                terms = f64(d[t]) * f64(y[pos[t, j]])
                want[t, j], tol[t, j] = terms.sum(), np.abs(terms).sum() * (Hd / 64 + 10) * U32
            H.close(f64(dw.t), want, tol, "f32", "dweights")
        assert dy.intact() and dw.intact()


U32 = 2.0 ** -24


def test_combine_grad_against_differences():
    """<dout, out> is linear in each weight: its difference quotient in 64
    bits equals dweights to the kernel's own rounding."""
    g = torch.Generator().manual_seed(0)
    y, d = torch.randn(6, 40, generator=g).cuda(), torch.randn(3, 40, generator=g).cuda()
    w = torch.rand(3, 2, generator=g).cuda()
    pos = torch.tensor([[0, 3], [5, -1], [2, 1]], dtype=torch.int32, device="cuda")
    dy, dw = torch.zeros(6, 40, device="cuda"), torch.zeros(3, 2, device="cuda")
    B.reshard_moe_combine_grad(B.MoeCombine("f32", "f32", 3, 2, 40, 6), ptr(d), ptr(y), ptr(pos), ptr(w), ptr(dy), ptr(dw), stream())
    p, yy, dd, ww = pos.cpu().numpy(), f64(y), f64(d), f64(w)
    base = (H.combine(yy, p, ww)[0] * dd).sum()
    for t in range(3):
        for j in range(2):
            up = ww.copy()
            up[t, j] += 1.0
            want = (H.combine(yy, p, up)[0] * dd).sum() - base
            assert abs(f64(dw)[t, j] - want) <= 40 * 12 * U32 * 8
    for r, c in ((0, 0), (3, 39), (4, 5), (1, 7)):
        up = yy.copy()
        up[r, c] += 1.0
        want = (H.combine(up, p, ww)[0] * dd).sum() - base
        assert abs(f64(dy)[r, c] - want) <= 8 * U32 + 1e-12 * abs(base)


# Groups whose experts do not divide evenly over a token's lanes: runs of up to 113 experts a lane.
WIDE_GROUPS = [(900, 9), (1020, 5), (1020, 6), (1000, 10), (771, 3), (585, 9), (1017, 9), (1023, 11), (1020, 12), (1014, 13),
               (1022, 14), (1020, 15), (1022, 7)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", WIDE_GROUPS)
def test_route_wide_groups(E, G, score):
    for dtype, biased, group_top, k in (("f32", True, 2, 8), ("f32", False, 2, 8), ("bf16", False, 1, 8), ("f16", True, 1, 17),
                                        ("f32", False, 1, 32)):
        x = logits_for(14, E, dtype, E + k)
        bias = (torch.randn(E, generator=torch.Generator().manual_seed(G)) * 0.05).cuda() if biased else None
        x[1, ::3] = -float("inf")
        x[2, : E - E // G] = float("nan")
        x[3] = 0.0   # all alike: the lowest groups and experts
        for renorm in (True, False):
            check_route(x, dict(k=k, score=score, renorm=renorm, groups=G, top_groups=(G + 1) // 2, group_top=group_top), bias,
                        dtype=dtype)


@pytest.mark.parametrize("E,G", [(900, 9), (771, 3)])
def test_route_wide_groups_take_the_last_experts(E, G):
    """Every expert of a group can be chosen, the last ones of a run too; near
    scores are told apart beyond float32."""
    x = torch.full((E, E), -3.0)
    x[torch.arange(E), torch.arange(E)] = 2.0
    x[torch.arange(E), (torch.arange(E) + E // G - 1) % E] = 1.0
    check_route(x.cuda(), dict(k=2, score="sigmoid", renorm=True, groups=G, top_groups=2))
    rng = np.random.default_rng(0)
    y = torch.tensor(rng.normal(0, 1, (40, E)), dtype=torch.float32)
    y[:, 1::2] = torch.nextafter(y[:, :-1:2], torch.full_like(y[:, :-1:2], 9.0))[:, : y[:, 1::2].shape[1]]
    for score in ("softmax", "sigmoid"):
        check_route(y.cuda(), dict(k=8, score=score, renorm=False, groups=G, top_groups=2, group_top=2), torch.full((E,), 0.4).cuda())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_of_saturated_sigmoids(dtype, renorm):
    """s (1 - s) keeps its digits where s is next to 1 as where it is next to
    0: e^-|l| / (1 + e^-|l|)^2 is off by 2 U from exp, the sum and the
    quotients by less than 8 U together, three products by 3 U; the
    renormalised weights' share (a second score, a sum over four slots, a
    quotient, the difference) by less than 40 U of the magnitudes subtracted."""
    x = torch.linspace(-80, 80, 64).repeat(16, 1)
    x[1::2] = torch.linspace(10, 40, 64)
    x = x.to(DT[dtype]).cuda()
    rng = np.random.default_rng(1)
    ids = np.stack([rng.permutation(64)[:4] for _ in range(16)]).astype(np.int32)
    ids[2] = [63, 60, 60, 62]
    g = rng.normal(0, 1, (16, 4)).astype(np.float32)
    r = B.Router(dtype, 64, 4, score="sigmoid", renormalise=renorm, scale=1.5)
    out = torch.full((16, 64), 7.0, dtype=DT[dtype], device="cuda")
    B.reshard_moe_route_grad(r, 16, ptr(x), 64, ptr(torch.from_numpy(ids).cuda()), ptr(torch.from_numpy(g).cuda()),
                             ptr(out), 64, stream())
    xx, want, tol = f64(x), np.zeros((16, 64)), np.zeros((16, 64))
    e = np.exp(-np.abs(xx))
    s, rest = np.where(xx >= 0, 1, e) / (1 + e), np.where(xx >= 0, e, 1) / (1 + e)   # rest = 1 - s
    for t in range(16):
        p = s[t, ids[t]]
        h = 1.5 * g[t].astype(np.float64)
        a = np.abs(h)
        if renorm:
            h, a = (h - (h * p).sum() / p.sum()) / p.sum(), (a + (a * p).sum() / p.sum()) / p.sum()
        for j in range(4):
            i = ids[t, j]
            want[t, i] += s[t, i] * rest[t, i] * h[j]
            tol[t, i] += s[t, i] * rest[t, i] * a[j] * (64 if renorm else 24) * H.U
    H.close(f64(out), want, tol, dtype, "dlogits")


def tiny_scores(score):
    """Logits and a bias that forces the choice of experts whose scores lie
    below the smallest normal float32 number, or below any."""
    x = torch.full((8, 16), 0.0)
    if score == "softmax":
        for t, d in enumerate((80.0, 95.0, 100.0, 110.0, 200.0, 600.0, 0.0, 30.0)):
            x[t, 8:] = d
    else:
        for t, d in enumerate((80.0, 88.5, 95.0, 100.0, 110.0, 200.0, 600.0, -3.0)):
            x[t, :8] = -d
    x[:, :8] += torch.linspace(-2, 2, 8)
    return x, torch.where(torch.arange(16) < 8, 2.0, 0.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [1, 4])
def test_route_renormalises_tiny_scores(score, k):
    x, bias = tiny_scores(score)
    for scale in (1.0, 2.5):
        check_route(x.cuda(), dict(k=k, score=score, renorm=True, scale=scale), bias.cuda())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_no_weight_where_the_scores_are_zero(score):
    """Sums that are 0 in double precision: logits below -745, next to one 800 or infinitely higher."""
    x, bias = tiny_scores(score)
    if score == "softmax":
        x[0, 8:], x[1, 8:], x[2, 8:] = 800.0, float("inf"), torch.finfo(torch.float32).max
    else:
        x[0, :8], x[1, :8], x[2, :8] = -800.0, -1e30, torch.finfo(torch.float32).min
    ids, w = run_route(x.cuda(), dict(k=3, score=score, renorm=True), bias.cuda())
    assert (w[:3] == 0).all() and (w[3:] > 0).all() and (ids < 8).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [1, 3])
def test_route_grad_of_tiny_scores(score, k):
    x, _ = tiny_scores(score)
    rng = np.random.default_rng(k)
    ids = np.stack([rng.permutation(8)[:k] for _ in range(8)]).astype(np.int32)
    g = rng.normal(0, 1, (8, k)).astype(np.float32)
    r = B.Router("f32", 16, k, score=score, renormalise=True, scale=2.0)
    out = torch.full((8, 16), 7.0, device="cuda")
    B.reshard_moe_route_grad(r, 8, ptr(x.cuda()), 16, ptr(torch.from_numpy(ids).cuda()), ptr(torch.from_numpy(g).cuda()),
                             ptr(out), 16, stream())
    want, tol = H.route_grad(f64(x), ids, g.astype(np.float64), dict(score=score, renorm=True, scale=2.0))
    H.close(f64(out), want, tol, "f32", "dlogits")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_token_does_not_depend_on_its_neighbours(score):
    """Ordinary tokens, tiny scores and equal ones in one wave give the bytes that each gives alone."""
    x, bias = tiny_scores(score)
    x = torch.cat([x, logits_for(29, 16, "f32", 5).cpu(), torch.zeros(3, 16)])[torch.randperm(40, generator=torch.Generator().manual_seed(0))]
    x, bias = x.cuda(), bias.cuda()
    c = dict(k=3, score=score, renorm=True)
    ids, w = run_route(x, c, bias)
    for t in range(40):
        i, v = run_route(x[t:t + 1], c, bias)
        assert torch.equal(ids[t:t + 1], i) and torch.equal(w[t:t + 1].view(torch.int32), v.view(torch.int32))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,group_top", [(1, 1), (4, 1), (4, 2), (3, 2)])
def test_route_bias_without_a_number(score, groups, group_top):
    """An expert whose bias is NaN or -infinity is never chosen and adds
    nothing to its group."""
    x = logits_for(40, 48, "f32", 12)
    bias = torch.randn(48, generator=torch.Generator().manual_seed(1)) * 0.1
    bias[2::3] = float("nan")
    if groups == 3:
        bias[[1, 16, 31]] = -float("inf")
    plain = torch.where(torch.isnan(bias), torch.full_like(bias, -float("inf")), bias)
    for k in (4, 14):
        c = dict(k=k, score=score, renorm=True, groups=groups, top_groups=(groups + 1) // 2, group_top=group_top)
        ids, w = run_route(x, c, bias.cuda())
        want, ww, tol = H.route(f64(x), c, f64(plain))
        assert np.array_equal(ids.cpu().numpy(), want)
        H.close(f64(w), ww, np.abs(ww) * tol[:, None], "f32", "weights")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_ignores_dweights_of_slots_without_a_score(score, renorm):
    x = logits_for(6, 32, "f32", 2)
    x[:, 5], x[:, 6] = -float("inf"), float("nan")
    ids = np.tile(np.array([[5, 1, 6, 2, -1, 32]], dtype=np.int32), (6, 1))
    dw = np.random.default_rng(0).normal(0, 1, (6, 6)).astype(np.float32)
    clean = dw.copy()
    clean[:, [0, 2, 4, 5]] = 0.0
    dw[:3, [0, 2, 4, 5]] = np.nan
    dw[3:, [0, 2, 4, 5]] = np.inf
    out = torch.full((6, 32), 7.0, device="cuda")
    B.reshard_moe_route_grad(B.Router("f32", 32, 6, score=score, renormalise=renorm), 6, ptr(x), 32, ptr(torch.from_numpy(ids).cuda()),
                             ptr(torch.from_numpy(dw).cuda()), ptr(out), 32, stream())
    want, tol = H.route_grad(f64(x), ids, clean.astype(np.float64), dict(score=score, renorm=renorm))
    H.close(f64(out), want, tol, "f32", "dlogits")


@pytest.mark.parametrize("E,G", [(512, 1), (1000, 1), (1024, 1), (1017, 9), (1020, 5)])
def test_route_where_the_sum_of_exponentials_rounds_one_way(E, G):
    """Many terms just above half a step of their sum: each addition rounds up,
    and the largest score comes out low by nearly as many steps.  Next to it
    stands an expert whose bias alone lies that near."""
    run = -(-E // 16) if G == 1 else E // G if G > 8 else -(-(E // G) // 2)   # experts a lane
    x = torch.full((10, E), -100.0)
    x[:, 0] = 0.0
    x[:, 1:run] = float(np.log(0.51 * 2.0 ** -23))
    s = 1 / (1 + np.exp(f64(x[0, 1:run])).sum())
    other = E // G - 1 if G > 1 else E - 1   # of the same group
    for gap in (-30, -2, 2, 10, 25, 40, 55, 100):
        bias = -10.0 - torch.arange(E) * 0.01
        bias[0] = -0.99
        bias[other] = float(np.float32(s + float(bias[0]) - gap * H.U))
        check_route(x.cuda(), dict(k=2, score="softmax", renorm=False, groups=G, top_groups=1), bias.cuda())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(16, 3), (128, 8), (1000, 20)])
def test_route_grad_of_a_score_next_to_one(score, renorm, E, k):
    """One expert far above the others: its own entry, s (1 - s) of the
    differences, keeps its digits.  Per expert, the scores are off as in
    H.route_grad; H (1 - s) - sum of the others' counts 3 U of each magnitude
    for the top one, H - sum of all three times what is left of it for the
    others (1 - s is a half there at the least)."""
    g = torch.Generator().manual_seed(E)
    x = torch.randn(12, E, generator=g) - (40 if score == "sigmoid" and renorm else 0)
    at = torch.arange(12) % E
    for t, gap in enumerate((0.5, 2, 5, 8, 10, 12, 14, 16, 18, 20, 25, 30)):
        x[t, at[t]] = x[t].max() + gap
    rng = np.random.default_rng(k)
    ids = np.stack([np.concatenate([[at[t]], rng.permutation(np.delete(np.arange(E), at[t]))[:k - 1]]) for t in range(12)]).astype(np.int32)
    ids = np.ascontiguousarray(np.take_along_axis(ids, np.argsort(rng.random(ids.shape), 1), 1))
    dw = rng.normal(0, 1, (12, k)).astype(np.float32)
    if k > 8:
        ids[::3, 0] = ids[::3, 1] = at[::3].numpy()   # named twice or more
    r = B.Router("f32", E, k, score=score, renormalise=renorm, scale=1.5)
    out = torch.full((12, E), 7.0, device="cuda")
    B.reshard_moe_route_grad(r, 12, ptr(x.cuda()), E, ptr(torch.from_numpy(ids).cuda()), ptr(torch.from_numpy(dw).cuda()), ptr(out), E, stream())
    s, d = H.scores(f64(x), score)
    want, tol = np.zeros((12, E)), np.zeros((12, E))
    for t in range(12):
        h, c = np.zeros(E), np.zeros(E)   # sums of dweights and of their magnitudes by expert, slots by expert
        a = np.zeros(E)
        for j in range(k):
            h[ids[t, j]] += 1.5 * dw[t, j]
            a[ids[t, j]] += 1.5 * abs(float(dw[t, j]))
            c[ids[t, j]] += 1
        if renorm:     # shares of the sum over the slots: sum_e c_e r_e = 1
            p = s[t] * (c > 0)
            w = p / (p * c).sum()
        else:
            w, c = s[t], np.ones(E)
        if not renorm and score == "sigmoid":
            e = np.exp(-np.abs(f64(x[t])))
            want[t], tol[t] = e / (1 + e) ** 2 * h, e / (1 + e) ** 2 * a * 24 * H.U
            continue
        # sum_f w_f (c_f h_e - c_e h_f), without cancellation of the part that e itself has
        diff, mag = np.zeros(E), np.zeros(E)
        for i in range(E):
            o = np.arange(E) != i
            diff[i] = h[i] * (w * c)[o].sum() - c[i] * (w * h)[o].sum()
            mag[i] = a[i] * (w * c)[o].sum() + c[i] * (w * a)[o].sum()
        f = 1 / (1 + np.exp(f64(x[t]))) if score == "sigmoid" else 1.0
        want[t], tol[t] = w * diff * f, w * mag * f * 3 * (2 * d[t] + 128 + k) * H.U
    H.close(f64(out), want, tol, "f32", "dlogits")
