"""Expert-FFN operators on rows so far apart that offsets pass 2^31 elements
and 2^32 bytes: only the rows' own elements are touched, so the large buffers
are never filled."""

import numpy as np
import pytest
import torch

from rl_weight_refit_amd import binding as B

import ops_helpers as H
from ops_helpers import U, f64, stream

pytestmark = pytest.mark.gpu

FAR = 1 << 30   # the largest stride


def ptr(t):   # the tests hold what they pass until they have read a result
    return None if t is None else t.data_ptr()


def far(rows, cols, stride, dtype):
    """rows x cols elements, stride apart, in memory that nothing fills."""
    whole = torch.empty((rows - 1) * stride + (cols + 15) // 16 * 16, dtype=dtype, device="cuda")
    return whole.as_strided((rows, cols), (stride, 1))


def placed(x, stride):
    t = far(x.shape[0], x.shape[1], stride, x.dtype)
    t.copy_(x)
    return t


def test_quantise_far_rows():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 300, generator=g).bfloat16()
    xd = placed(x, FAR)
    for kw, rows, cols, want in ((dict(), 5, 300, H.quantise(f64(x), 1)), (dict(block_rows=128), 5, 300, H.quantise(f64(x), 128))):
        q = far(rows, cols, FAR, torch.uint8)
        s = torch.empty(want[1].shape, device="cuda")
        d = B.Fp8Quant("bf16", rows, cols, x_stride=FAR, code_stride=FAR, **kw)
        B.reshard_fp8_quantise(d, ptr(xd), None, ptr(q), ptr(s), stream())
        assert np.array_equal(q.cpu().numpy(), want[0]) and np.array_equal(s.cpu().numpy(), want[1])


# The large tiles' load offsets are 32 bits: 2^23 bytes apart a tile's rows lie
# within them and the tiles' beginnings beyond; 2^24 - 16 apart a tile's last rows
# lie beyond 2^31.  With an index all of a would have to lie within.
@pytest.mark.parametrize("rows,stride,index", [(600, 1 << 23, False), (260, (1 << 24) - 16, False), (600, 1 << 23, True),
                                               (5, FAR, False), (5, FAR, True)])
@pytest.mark.parametrize("side", ["a", "b", "c"])
def test_matmul_far_rows(rows, stride, index, side):
    rng = np.random.default_rng(rows)
    M, N, K = (rows, 320, 272) if side != "b" else (320, rows, 272)
    codes = [torch.from_numpy(H.random_codes(rng, r, K)) for r in (M, N)]
    scales = [rng.uniform(0.5, 2.0, (r, 3)).astype(np.float32) for r in (M, N)]
    values = [H.mxfp8.e4m3_decode(c.numpy()) * np.repeat(s.astype(np.float64), 128, 1)[:, :K] for c, s in zip(codes, scales)]
    a, b = (placed(c, stride if side == n else K) if side == n else c.cuda() for c, n in zip(codes, "ab"))
    order = rng.integers(0, M, M).astype(np.int32) if index else np.arange(M)
    c = far(M, N, stride // 2, torch.bfloat16) if side == "c" else torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    mm = B.Fp8Matmul(M, N, K, "bf16", a_stride=stride if side == "a" else K, b_stride=stride if side == "b" else K,
                     b_block_rows=1, c_stride=c.stride(0))
    idx = torch.from_numpy(order).cuda() if index else None
    sa, sb = (torch.from_numpy(s).cuda() for s in scales)
    B.reshard_fp8_matmul(mm, ptr(a), ptr(sa), ptr(idx), ptr(b), ptr(sb), None, ptr(c), stream())
    want, tol = H.product(values[0][order], values[1], 3, "bf16")
    H.close(f64(c.contiguous()), want, tol, "bf16", "c")


def test_combine_far_rows():
    g = torch.Generator().manual_seed(1)
    T, k, Hd, rows = 5, 2, 200, 5
    y, d, w = torch.randn(rows, Hd, generator=g).bfloat16(), torch.randn(T, Hd, generator=g).bfloat16(), torch.rand(T, k, generator=g)
    pos = np.array([[4, -1], [0, 3], [-1, -1], [1, -1], [-1, 2]], dtype=np.int32)
    desc = B.MoeCombine("bf16", "bf16", T, k, Hd, rows, y_stride=FAR, out_stride=FAR)
    yd, dd, out, dy = placed(y, FAR), placed(d, FAR), far(T, Hd, FAR, torch.bfloat16), far(rows, Hd, FAR, torch.bfloat16)
    pd, wd, dw = torch.from_numpy(pos).cuda(), w.cuda(), torch.empty(T, k, device="cuda")
    B.reshard_moe_combine(desc, ptr(yd), ptr(pd), ptr(wd), ptr(out), stream())
    B.reshard_moe_combine_grad(desc, ptr(dd), ptr(yd), ptr(pd), ptr(wd), ptr(dy), ptr(dw), stream())
    want, wdy, wdw, mag = np.zeros((T, Hd)), np.zeros((rows, Hd)), np.zeros((T, k)), np.zeros((T, k))
    for t, j in zip(*np.nonzero(pos >= 0)):
        want[t] += f64(w)[t, j] * f64(y)[pos[t, j]]
        wdy[pos[t, j]] = f64(w)[t, j] * f64(d)[t]
        terms = f64(d)[t] * f64(y)[pos[t, j]]
        wdw[t, j], mag[t, j] = terms.sum(), np.abs(terms).sum()
    # at most two products and an addition, then the rounding to bf16
    room = np.zeros((T, Hd))
    for t, j in zip(*np.nonzero(pos >= 0)):
        room[t] += 3 * U * np.abs(f64(w)[t, j] * f64(y)[pos[t, j]])
    H.close(f64(out.contiguous()), want, room, "bf16", "out")
    H.close(f64(dy.contiguous()), wdy, np.abs(wdy) * U, "bf16", "dy")
    H.close(f64(dw), wdw, mag * (Hd / 64 + 10) * U, "f32", "dweights")


def test_route_far_rows():
    g = torch.Generator().manual_seed(2)
    T, E, k = 5, 64, 4
    x = torch.randn(T, E, generator=g).bfloat16()
    xd, dl = placed(x, FAR), far(T, E, FAR, torch.bfloat16)
    near, dn = x.cuda(), torch.empty(T, E, dtype=torch.bfloat16, device="cuda")
    r = B.Router("bf16", E, k)
    got = []
    for t, stride in ((xd, FAR), (near, E)):
        ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
        B.reshard_moe_route(r, T, ptr(t), stride, None, None, ptr(ids), ptr(w), stream())
        out = dl if stride == FAR else dn
        B.reshard_moe_route_grad(r, T, ptr(t), stride, ptr(ids), ptr(w), ptr(out), stride, stream())
        got.append((ids.cpu(), w.cpu(), out.contiguous().cpu()))
    assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(*got))


# What the tiles' 32-bit offsets do not reach: gathered rows spread over 4 GiB or more, and rows of either side (or their
# scales) so far apart that one tile's span as much.
@pytest.mark.parametrize("side,rows,stride", [("a gathered", 4200, 1 << 20), ("a gathered", 9000, 1 << 19), ("a", 150, 1 << 25),
                                              ("b", 150, 1 << 25), ("a scales", 150, 1 << 23), ("b scales", 330, 1 << 22)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_matmul_tiles_beyond_32_bit_offsets(side, rows, stride, out):
    rng = np.random.default_rng(rows)
    M, N, K = (rows, 300, 408) if side[0] == "a" else (320, rows, 408)
    codes = [torch.from_numpy(H.random_codes(rng, r, 416)) for r in (M, N)]
    scales = [torch.from_numpy(rng.uniform(0.5, 2.0, (r, 4)).astype(np.float32)) for r in (M, N)]
    values = [H.mxfp8.e4m3_decode(c.numpy()) * np.repeat(f64(s), 128, 1)[:, :416] for c, s in zip(codes, scales)]
    a, b = (placed(t, stride) if name in (side, side[:-9]) else t.cuda() for t, name in zip(codes, "ab"))
    sa, sb = (placed(t, stride) if name + " scales" == side else t.cuda() for t, name in zip(scales, "ab"))
    order = rng.integers(-1, M + 1, 700).astype(np.int32) if side == "a gathered" else np.arange(M, dtype=np.int32)
    order[:2] = [M - 1, 0]
    idx = torch.from_numpy(order).cuda() if side == "a gathered" else None
    if idx is None:
        order = np.arange(M)
    c = torch.zeros(len(order), N, dtype=H.DT[out], device="cuda")
    mm = B.Fp8Matmul(len(order), N, K, out, a_rows=M, a_stride=a.stride(0), a_scale_stride=sa.stride(0), b_stride=b.stride(0),
                     b_scale_stride=sb.stride(0), b_block_rows=1)
    B.reshard_fp8_matmul(mm, ptr(a), ptr(sa), ptr(idx), ptr(b), ptr(sb), None, ptr(c), stream())
    av = np.where(((order >= 0) & (order < M))[:, None], values[0][np.clip(order, 0, M - 1)], 0.0)
    want, tol = H.product(av[:, :K], values[1][:, :K], 4, out)
    H.close(f64(c), want, tol, out, "c")


def test_matmul_far_gathered_groups():
    rng = np.random.default_rng(3)
    M, N, K, rows = 300, 256, 256, 4200
    a, sa = torch.from_numpy(H.random_codes(rng, rows, K)), rng.uniform(0.5, 2.0, (rows, 2)).astype(np.float32)
    b, sb = torch.from_numpy(H.random_codes(rng, 2 * N, K)), rng.uniform(0.5, 2.0, (2, 2, 2)).astype(np.float32)
    far_a = placed(a, 1 << 20)
    far_b = torch.empty((1 << 32) + N * K, dtype=torch.uint8, device="cuda").as_strided((2, N, K), (1 << 32, K, 1))
    far_b.copy_(b.view(2, N, K))
    off, idx = np.array([0, 170, 300], dtype=np.int32), rng.integers(0, rows, M).astype(np.int32)
    c = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    mm = B.Fp8Matmul(M, N, K, "bf16", groups=2, a_rows=rows, a_stride=1 << 20, b_group_stride=1 << 32)
    dev = [torch.from_numpy(v).cuda() for v in (sa, idx, sb, off)]
    B.reshard_fp8_matmul(mm, ptr(far_a), ptr(dev[0]), ptr(dev[1]), ptr(far_b), ptr(dev[2]), ptr(dev[3]), ptr(c), stream())
    av = (H.mxfp8.e4m3_decode(a.numpy()) * np.repeat(sa.astype(np.float64), 128, 1))[idx]
    bv = H.mxfp8.e4m3_decode(b.numpy()).reshape(2, N, K) * np.repeat(np.repeat(sb.astype(np.float64), 128, 1), 128, 2)
    for g in range(2):
        want, tol = H.product(av[off[g]:off[g + 1]], bv[g], 2, "bf16")
        H.close(f64(c[off[g]:off[g + 1]]), want, tol, "bf16", "group %d" % g)


def test_matmul_far_gathered_rows_in_one_launch():
    """2.2 million rows gathered from 4 GiB, by 4096 columns: 550,000 tiles of
    64 x 256, where one of 32 x 32 each would take more threads than a launch
    holds."""
    rng = np.random.default_rng(4)
    M, N, K, rows = 2_200_000, 4096, 128, 4200
    a, sa = torch.from_numpy(H.random_codes(rng, rows, K)), rng.uniform(0.5, 2.0, (rows, 1)).astype(np.float32)
    b, sb = torch.from_numpy(H.random_codes(rng, N, K)), rng.uniform(0.5, 2.0, (N // 128, 1)).astype(np.float32)
    idx = rng.integers(0, rows, M).astype(np.int32)
    far_a, c = placed(a, 1 << 20), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    dev = [torch.from_numpy(v).cuda() for v in (sa, idx, sb)]
    bd = b.cuda()
    mm = B.Fp8Matmul(M, N, K, "bf16", a_rows=rows, a_stride=1 << 20)
    B.reshard_fp8_matmul(mm, ptr(far_a), ptr(dev[0]), ptr(dev[1]), ptr(bd), ptr(dev[2]), None, ptr(c), stream())
    some = np.concatenate([np.arange(70), np.arange(M - 70, M), rng.integers(0, M, 400)])
    av = (H.mxfp8.e4m3_decode(a.numpy()) * sa.astype(np.float64))[idx[some]]
    want, tol = H.product(av, H.mxfp8.e4m3_decode(b.numpy()) * np.repeat(sb.astype(np.float64), 128, 0), 1, "bf16")
    H.close(f64(c[torch.from_numpy(some).cuda()]), want, tol, "bf16", "c")


def test_sort_of_the_most_slots():
    """2^30 slots, against a stable sort."""
    T, k, E, first, local = 1 << 27, 8, 40, 5, 30
    ids = torch.randint(-1, E, (T, k), dtype=torch.int32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0))
    off = torch.empty(local + 1, dtype=torch.int32, device="cuda")
    tok, pos = torch.empty(T * k, dtype=torch.int32, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    ws = torch.empty(B.reshard_moe_sort_workspace(T, k, local), dtype=torch.uint8, device="cuda")
    B.reshard_moe_sort(ptr(ids), T, k, first, local, ptr(off), ptr(tok), ptr(pos), ptr(ws), ws.numel(), stream())
    e = ids.view(-1) - first
    e = torch.where((e >= 0) & (e < local), e, local)
    counts = torch.bincount(e, minlength=local + 1)
    want = torch.zeros(local + 1, dtype=torch.int64, device="cuda")
    want[1:] = counts[:local].cumsum(0)
    assert torch.equal(off.long(), want)
    rows = int(want[-1])
    order = torch.sort(e.to(torch.uint8), stable=True).indices[:rows]
    assert torch.equal(pos.view(-1)[order], torch.arange(rows, dtype=torch.int32, device="cuda"))
    assert torch.equal(tok[:rows], torch.div(order, k, rounding_mode="floor").int()) and bool((tok[rows:] == -1).all())
    assert int((pos == -1).sum()) == T * k - rows


def test_quantise_a_row_of_the_most_columns():
    """One row of 2^31 values has the codes of 2^24 rows of 128."""
    n = 1 << 31
    x = torch.randn(1 << 20, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0)).bfloat16().repeat(16, 1)
    x[-1] *= 7
    got = []
    for rows, cols in ((1, n), (n // 128, 128)):
        q, s = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty(n // 128, device="cuda")
        B.reshard_fp8_quantise(B.Fp8Quant("bf16", rows, cols), ptr(x), None, ptr(q), ptr(s), stream())
        got.append((q, s))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    want = H.quantise(x[-300:].float().cpu().numpy(), 1)
    assert np.array_equal(got[0][0][-300 * 128:].cpu().numpy(), want[0].reshape(-1)) and np.array_equal(got[0][1][-300:].cpu().numpy(), want[1][:, 0])


def test_combine_wide_rows():
    """Rows of more than 65,535 workgroups of 2048 columns."""
    n = (1 << 27) + (1 << 24) + 5
    g = torch.Generator(device="cuda").manual_seed(0)
    y = torch.randn(3, n, device="cuda", generator=g).bfloat16()
    pos, w = torch.tensor([[2, 0], [-1, 1]], dtype=torch.int32, device="cuda"), torch.tensor([[0.5, 3.0], [1.0, -0.75]], device="cuda")
    out = torch.empty(2, n, dtype=torch.bfloat16, device="cuda")
    B.reshard_moe_combine(B.MoeCombine("bf16", "bf16", 2, 2, n, 3), ptr(y), ptr(pos), ptr(w), ptr(out), stream())
    # half, -3/4 and thrice of a bf16 value are exact in float32, and so is one rounding of their sum in float64
    assert torch.equal(out[1], (y[1].float() * -0.75).bfloat16())
    want = y[2].double() * 0.5 + y[0].double() * 3.0
    assert bool(((out[0].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -24) + 1e-38).all())


def test_route_of_many_tokens():
    """Row offsets beyond 2^31 elements."""
    T, E = (1 << 25) + 3, 72
    x = torch.randn(1 << 16, E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0)).bfloat16()
    whole = torch.empty(T, E, dtype=torch.bfloat16, device="cuda")
    whole[: 1 << 25].view(512, 1 << 16, E).copy_(x)
    whole[1 << 25:] = x[:3]
    r = B.Router("bf16", E, 3, score="sigmoid")
    got = []
    for t in (whole, x):
        ids, w = torch.empty(t.shape[0], 3, dtype=torch.int32, device="cuda"), torch.empty(t.shape[0], 3, device="cuda")
        B.reshard_moe_route(r, t.shape[0], ptr(t), E, None, None, ptr(ids), ptr(w), stream())
        dl = torch.empty_like(t)
        B.reshard_moe_route_grad(r, t.shape[0], ptr(t), E, ptr(ids), ptr(w), ptr(dl), E, stream())
        got.append((ids, w, dl))
    for a, b in zip(*got):
        assert torch.equal(a[: 1 << 25].view(512, 1 << 16, -1), b.expand(512, -1, -1)) and torch.equal(a[1 << 25:], b[:3])
