"""Block-FP8 quantisation and products on the GPU against plain 64-bit forms."""

import numpy as np
import pytest
import torch

import matmul_shapes
import ops_helpers as H
from ops_helpers import B, DT, Guarded, f64, ptr, stream, strided

pytestmark = pytest.mark.gpu


def run_quantise(x, dtype, rows, cols, pad=0, row_count=None, **kw):
    """Codes and scales of x (2-D device tensor) through padded, poisoned buffers."""
    orows, ocols = (cols, rows) if kw.get("transpose") else (rows, cols)
    srows = orows if kw.get("block_rows", 1) == 1 else -(-orows // 128)
    xs = strided(x, x.shape[1] + pad, pad)
    q, s = Guarded(orows, ocols, torch.uint8, ocols + pad, pad), Guarded(srows, -(-ocols // 128), torch.float32, -(-ocols // 128) + pad, pad)
    d = B.Fp8Quant(dtype, rows, cols, x_stride=xs.stride, code_stride=q.stride, scale_stride=s.stride, **kw)
    B.reshard_fp8_quantise(d, xs.ptr, ptr(row_count), q.ptr, s.ptr, stream())
    torch.cuda.synchronize()
    assert q.intact() and s.intact() and xs.intact()
    return q.t.cpu().numpy(), s.t.cpu().numpy()


SIZES = [(1, 1), (1, 128), (3, 130), (128, 128), (129, 127), (200, 520), (77, 1000), (5, 7168), (260, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantise(dtype, block_rows, transpose, rows, cols):
    g = torch.Generator().manual_seed(rows + cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))).to(DT[dtype])
    x[0, 0] = -0.0
    want = H.quantise(x.float().numpy().T if transpose else x.float().numpy(), block_rows)
    for pad in (0, 8, 3):
        q, s = run_quantise(x.cuda(), dtype, rows, cols, pad, block_rows=block_rows, transpose=transpose)
        assert np.array_equal(s.view(np.uint32), want[1].view(np.uint32))
        assert np.array_equal(q, want[0])


@pytest.mark.parametrize("block_rows,transpose", [(1, False), (1, True), (128, False), (128, True)])
def test_quantise_special_blocks(block_rows, transpose):
    """Zero blocks, scales below the smallest normal, the largest values, NaN and infinities."""
    x = torch.randn(260, 640, generator=torch.Generator().manual_seed(3))
    x[:, 128:256] = 0.0
    x[:, 128] = -0.0
    x[:130, 256:384] = 1e-37
    x[130:, 256:384] = 6e-36
    x[3, 400] = float("nan")
    x[200, 390] = float("inf")
    x[5, 520] = -float("inf")
    x[17, 600] = torch.finfo(torch.float32).max
    x[18, 601] = -torch.finfo(torch.float32).max
    want = H.quantise(x.numpy().T if transpose else x.numpy(), block_rows)
    q, s = run_quantise(x.cuda(), "f32", 260, 640, block_rows=block_rows, transpose=transpose)
    assert np.array_equal(np.isnan(s), np.isnan(want[1]))
    ok = ~np.isnan(s)
    assert np.array_equal(s[ok].view(np.uint32), want[1][ok].view(np.uint32))
    assert np.array_equal(q, want[0])


def test_quantise_every_bf16_value():
    """Every finite bf16 value once, next to a fixed largest value per row."""
    bits = np.arange(65536, dtype=np.uint16)
    v = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
    v = v[torch.isfinite(v.float())]
    n = v.numel() // 127 * 127
    for top in (1.0, 448.0, 3.0e38, 1.0e-30):
        x = torch.full((n // 127, 128), top, dtype=torch.bfloat16)
        x[:, 1:] = v[:n].view(-1, 127)
        want = H.quantise(x.float().numpy(), 1)
        q, s = run_quantise(x.cuda(), "bf16", x.shape[0], 128)
        assert np.array_equal(s.view(np.uint32), want[1].view(np.uint32))
        assert np.array_equal(q, want[0])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 384), (130, 200), (33, 515)])
def test_quantise_gated(dtype, transpose, rows, cols):
    """silu(gate) * up: the scale follows the 64-bit value to float32's
    rounding (exp, a quotient and three products: below 8 U), every code is
    the nearest to within that."""
    g = torch.Generator().manual_seed(rows)
    x = (torch.randn(rows, 2 * cols, generator=g) * 3).to(DT[dtype])
    gate, up = f64(x[:, :cols]), f64(x[:, cols:])
    v = gate / (1 + np.exp(-gate)) * up
    v = v.T if transpose else v
    for pad in (0, 8, 3):
        q, s = run_quantise(x.cuda(), dtype, rows, cols, pad, gated=True, transpose=transpose)
        M, K = v.shape
        for b in range(-(-K // 128)):
            at = np.abs(v[:, b * 128:(b + 1) * 128]).max(1) / 448
            H.close(s[:, b], at, at * 10 * H.U, "f32", "scales")
        sc = H.spread(s, 1, M, K)
        got = H.mxfp8.e4m3_decode(q) * sc
        # half a step of E4M3: 2^-4 of the value, or 2^-10 scales below the normal range
        room = np.maximum(np.abs(v) * 2.0 ** -4, sc * 2.0 ** -10) * (1 + 2.0 ** -10) + np.abs(v) * 16 * H.U
        assert (np.abs(got - v) <= room).all()


def test_quantise_gated_special_values():
    """A gate of -infinity times zero, an overflowing product: their block is marked."""
    x = torch.randn(4, 512, generator=torch.Generator().manual_seed(1))
    x[0, 3] = -float("inf")
    x[1, 5], x[1, 256 + 5] = 3e38, 3e38
    x[2, 7] = -1e30          # silu is -0
    x[3, 9], x[3, 256 + 9] = 100.0, 1e-30
    q, s = run_quantise(x.cuda(), "f32", 4, 256, gated=True)
    assert np.isnan(s[:2, 0]).all() and (q[:2, :128] == 0x7F).all()
    assert np.isfinite(s[2:]).all() and np.isfinite(s[:2, 1]).all()
    assert q[2, 7] in (0x00, 0x80)


def test_quantise_stops_at_the_row_count():
    x = torch.randn(50, 300, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    want = H.quantise(f64(x), 1)
    for n in (0, 1, 17, 50, 60, -3):
        q, s = run_quantise(x, "bf16", 50, 300, row_count=torch.tensor([n], dtype=torch.int32, device="cuda"))
        m = max(0, min(n, 50))
        assert np.array_equal(q[:m], want[0][:m]) and (q[m:] == 0xA5).all()
        assert np.array_equal(s[:m], want[1][:m]) and (s[m:].view(np.uint32) == 0xA5A5A5A5).all()


@pytest.mark.parametrize("block_rows,transpose", [(1, False), (1, True), (128, False), (128, True)])
def test_quantise_batch(block_rows, transpose):
    x = torch.randn(3, 200, 144, generator=torch.Generator().manual_seed(1)).bfloat16()
    d = B.Fp8Quant("bf16", 200, 144, batch=3, block_rows=block_rows, transpose=transpose)
    want = [H.quantise(f64(m).T if transpose else f64(m), block_rows) for m in x]
    q = torch.zeros(3, *want[0][0].shape, dtype=torch.uint8, device="cuda")
    s = torch.zeros(3, *want[0][1].shape, device="cuda")
    B.reshard_fp8_quantise(d, ptr(x.cuda()), None, ptr(q), ptr(s), stream())
    for i in range(3):
        assert np.array_equal(q[i].cpu().numpy(), want[i][0]) and np.array_equal(s[i].cpu().numpy(), want[i][1])


def test_quantise_nothing():
    B.reshard_fp8_quantise(B.Fp8Quant("bf16", 0, 128), None, None, None, None, stream())
    B.reshard_fp8_quantise(B.Fp8Quant("bf16", 4, 0), None, None, None, None, stream())


# --- products ---------------------------------------------------------------

def up16(n):
    return -(-n // 16) * 16


class Operand:
    """Random codes [G, R, K] with poisoned (NaN) padding behind each row, and scales."""

    def __init__(self, rng, G, R, K, block_rows, pad=0, split=0, factor=1.0):
        self.codes = H.random_codes(rng, G * R, K).reshape(G, R, K)
        srows = R if block_rows == 1 else (-(-split // 128) + -(-(R - split) // 128))
        self.scales = (rng.uniform(0.5, 2.0, (G, srows, -(-K // 128))) * factor).astype(np.float32)
        self.ld = up16(K) + pad
        raw = np.full((G, R, self.ld), 0x7F, dtype=np.uint8)
        raw[:, :, :K] = self.codes
        self.dev = torch.from_numpy(raw).cuda()
        self.sdev = torch.from_numpy(self.scales).cuda()
        n = np.arange(R)
        block = n if block_rows == 1 else np.where(n < split, n // 128, -(-split // 128) + (n - split) // 128) if split else n // 128
        self.values = H.mxfp8.e4m3_decode(self.codes) * np.repeat(self.scales[:, block].astype(np.float64), 128, 2)[:, :, :K]


def check_matmul(M, N, K, out="bf16", groups=None, b_rows=128, index_rows=0, split=0, pad=0, c_pad=0, seed=0, tail=0,
                 factor=1.0):
    """groups: rows per group; tail: rows behind the last group."""
    rng = np.random.default_rng(seed)
    G = len(groups) if groups else 0
    if groups:
        M = sum(groups) + tail
    rows = index_rows or M
    a, b = Operand(rng, 1, rows, K, 1, pad, factor=factor), Operand(rng, max(1, G), N, K, b_rows, pad, split)
    index = None
    if index_rows:
        idx = rng.integers(0, rows, M).astype(np.int32)
        if M > 3:
            idx[1], idx[2], idx[3] = -1, rows, -2 ** 31
        index = torch.from_numpy(idx).cuda()
        av = np.where(((idx >= 0) & (idx < rows))[:, None], a.values[0][np.clip(idx, 0, rows - 1)], 0.0)
    else:
        av = a.values[0]
    offsets, off = None, None
    if groups:
        off = np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)
        offsets = torch.from_numpy(off).cuda()
    c = Guarded(M, N, DT[out], N + c_pad, c_pad)
    before = c.t.clone()
    mm = B.Fp8Matmul(M, N, K, out, groups=G, a_rows=rows, a_stride=a.ld, b_stride=b.ld, b_block_rows=b_rows,
                     b_split=split, c_stride=c.stride)
    B.reshard_fp8_matmul(mm, ptr(a.dev), ptr(a.sdev), ptr(index), ptr(b.dev), ptr(b.sdev), ptr(offsets), c.ptr, stream())
    torch.cuda.synchronize()
    kb = -(-K // 128)
    got = f64(c.t)
    if not groups:
        want, tol = H.product(av, b.values[0], kb, out)
        H.close(got, want, tol, out, "c")
    else:
        for g in range(G):
            want, tol = H.product(av[off[g]:off[g + 1]], b.values[g], kb, out)
            H.close(got[off[g]:off[g + 1]], want, tol, out, "group %d" % g)
        assert torch.equal(c.t[off[-1]:].contiguous().view(torch.uint8), before[off[-1]:].contiguous().view(torch.uint8))
    assert c.intact()


MATMULS = [(1, 1, 1), (1, 128, 128), (1, 1000, 1333), (2, 64, 16), (7, 129, 300), (16, 256, 4096), (17, 200, 640), (33, 384, 17),
           (64, 64, 128), (65, 63, 129), (100, 257, 1000), (128, 512, 256), (130, 130, 130), (250, 300, 520),
           (256, 256, 512), (257, 513, 260), (300, 1024, 1024), (513, 640, 384), (1000, 768, 896)]


@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("M,N,K", MATMULS)
def test_matmul(M, N, K, b_rows):
    # float32 out shows the sums themselves, the others their rounding
    check_matmul(M, N, K, "f32", b_rows=b_rows, seed=M)
    check_matmul(M, N, K, "bf16", b_rows=b_rows, pad=48, c_pad=3, seed=N)


@pytest.mark.parametrize("M,N,K", [(5, 40, 200), (130, 200, 384), (300, 520, 256)])
def test_matmul_f16_out(M, N, K):
    check_matmul(M, N, K, "f16", seed=K)                     # most sums overflow
    check_matmul(M, N, K, "f16", seed=K, factor=2.0 ** -9)   # none does


@pytest.mark.parametrize("M,N,K", [(1, 48, 300), (40, 130, 128), (260, 256, 400), (700, 300, 256)])
@pytest.mark.parametrize("rows", [1, 33, 500])
def test_matmul_gathers_rows(M, N, K, rows):
    check_matmul(M, N, K, "f32", index_rows=rows, seed=M + rows)


GROUPS = [[1], [0, 0, 0], [3, 0, 5], [0, 64, 1, 0, 65, 130], [16] * 8, [1] * 70, [300, 0, 2, 17], [0] * 130 + [9],
          [257, 511, 1, 64], [5, 700, 3]]


@pytest.mark.parametrize("which", range(len(GROUPS)))
@pytest.mark.parametrize("b_rows", [128, 1])
def test_matmul_groups(which, b_rows):
    check_matmul(0, 200, 392, "f32", groups=GROUPS[which], b_rows=b_rows, seed=which, tail=which % 3 * 40)
    check_matmul(0, 256, 256, "bf16", groups=GROUPS[which], b_rows=b_rows, seed=which, index_rows=50, tail=7)


# As many tiles as fill the chip: 256, 128, 64 rows by 256 columns.
@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(2900, 3000, 392), (1900, 3000, 392), (1000, 3000, 4000)])
def test_matmul_many_tiles(M, N, K, out, b_rows):
    check_matmul(M, N, K, out, b_rows=b_rows, c_pad=5, seed=M)


@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("K", [256, 392, 100])
def test_matmul_many_tiles_in_groups(out, b_rows, K):
    """Tiles of 256 rows, whole ones, some with half their rows or fewer, absent ones."""
    check_matmul(0, 3000, K, out, b_rows=b_rows, groups=[1500, 129, 0, 1, 900, 128, 257, 60, 1330], index_rows=500, tail=9,
                 seed=K)


@pytest.mark.parametrize("N,split", [(256, 128), (200, 100), (600, 300), (96, 48), (513, 257), (300, 1), (512, 320)])
def test_matmul_two_part_scales(N, split):
    """Gate and up rows of a fused w13 whose halves are not whole scale blocks."""
    check_matmul(70, N, 384, "f32", split=split)
    check_matmul(0, N, 256, "bf16", groups=[5, 0, 150, 40], split=split)
    check_matmul(3, N, 256, "bf16", split=split)


def test_matmul_nan_codes_stay_in_their_rows():
    """A NaN code of a reaches its row of c only, one of b its column only."""
    rng = np.random.default_rng(0)
    for M, N, K in ((40, 80, 300), (300, 512, 512), (3, 256, 384)):
        a, b = Operand(rng, 1, M, K, 1), Operand(rng, 1, N, K, 128)
        a.dev[0, 1, 5] = 0x7F
        b.dev[0, 7, K - 1] = 0xFF
        c = torch.zeros(M, N, device="cuda")
        mm = B.Fp8Matmul(M, N, K, "f32", a_stride=a.ld, b_stride=b.ld)
        B.reshard_fp8_matmul(mm, ptr(a.dev), ptr(a.sdev), None, ptr(b.dev), ptr(b.sdev), None, ptr(c), stream())
        want = torch.zeros(M, N, dtype=torch.bool)
        want[1] = True
        want[:, 7] = True
        assert torch.equal(torch.isnan(c).cpu(), want)


def test_matmul_nothing_and_empty_k():
    B.reshard_fp8_matmul(B.Fp8Matmul(0, 16, 16, "f32"), None, None, None, None, None, None, None, stream())
    B.reshard_fp8_matmul(B.Fp8Matmul(4, 0, 16, "f32"), None, None, None, None, None, None, None, stream())
    c = torch.full((3, 5), 7.0, device="cuda")
    B.reshard_fp8_matmul(B.Fp8Matmul(3, 5, 0, "f32"), None, None, None, None, None, None, ptr(c), stream())
    assert (c == 0).all()


def test_matmul_offsets_out_of_range_write_nothing_outside():
    """Offsets beyond m are cut to it; descending ones give empty groups."""
    rng = np.random.default_rng(0)
    a, b = Operand(rng, 1, 40, 128, 1), Operand(rng, 3, 64, 128, 128)
    for off, rows in (([0, 30, 50, 90], 40), ([5, 10, 10, 20], 15), ([0, 30, 20, 25], 35), ([-7, 3, 3, 3], 3)):
        c = Guarded(40, 64, torch.float32)
        mm = B.Fp8Matmul(40, 64, 128, "f32", groups=3, a_stride=a.ld, b_stride=b.ld)
        B.reshard_fp8_matmul(mm, ptr(a.dev), ptr(a.sdev), None, ptr(b.dev), ptr(b.sdev),
                             ptr(torch.tensor(off, dtype=torch.int32, device="cuda")), c.ptr, stream())
        torch.cuda.synchronize()
        assert c.intact()


def test_linear_layer_forward_and_both_gradients():
    """y = x W^T, dx = dy W and dW = dy^T x through the quantiser's modes: each
    product equals the 64-bit product of what was quantised, and what was
    quantised is within E4M3's half step (2^-4, or 2^-10 scales) of the
    input."""
    g = torch.Generator().manual_seed(0)
    M, N, K = 200, 320, 272
    x, w, dy = (torch.randn(*s, generator=g).bfloat16().cuda() for s in ((M, K), (N, K), (M, N)))

    def quantise(v, **kw):
        rows, cols = v.shape
        orows, ocols = (cols, rows) if kw.get("transpose") else (rows, cols)
        q = torch.zeros(orows, up16(ocols), dtype=torch.uint8, device="cuda")
        s = torch.zeros(orows if kw.get("block_rows", 1) == 1 else -(-orows // 128), -(-ocols // 128), device="cuda")
        B.reshard_fp8_quantise(B.Fp8Quant("bf16", rows, cols, code_stride=q.shape[1], **kw), ptr(v), None, ptr(q), ptr(s), stream())
        back = H.values(q[:, :ocols].cpu().numpy(), s.cpu().numpy(), kw.get("block_rows", 1))
        want = f64(v).T if kw.get("transpose") else f64(v)
        room = np.maximum(np.abs(want) * 2.0 ** -4, H.spread(s.cpu().numpy(), kw.get("block_rows", 1), orows, ocols) * 2.0 ** -10)
        assert (np.abs(back - want) <= room * (1 + 2.0 ** -10)).all()
        return q, s, back

    def product(a, b, b_rows, n_k):
        (qa, sa, va), (qb, sb, vb) = a, b
        c = torch.zeros(va.shape[0], vb.shape[0], device="cuda")
        mm = B.Fp8Matmul(va.shape[0], vb.shape[0], n_k, "f32", a_stride=qa.shape[1], b_stride=qb.shape[1], b_block_rows=b_rows)
        B.reshard_fp8_matmul(mm, ptr(qa), ptr(sa), None, ptr(qb), ptr(sb), None, ptr(c), stream())
        want, tol = H.product(va, vb, -(-n_k // 128), "f32")
        H.close(f64(c), want, tol, "f32", "product")
        return f64(c)

    wq = quantise(w, block_rows=128)
    wt = quantise(w, block_rows=128, transpose=True)
    assert np.array_equal(wq[2], wt[2].T)   # 128 x 128 blocks quantise alike either way round
    product(quantise(x), wq, 128, K)
    product(quantise(dy), wt, 128, N)
    product(quantise(dy, transpose=True), quantise(x, transpose=True), 1, M)


@pytest.mark.parametrize("block_rows,transpose", [(1, False), (1, True), (128, False), (128, True)])
def test_quantise_gated_small_sigmoids(block_rows, transpose):
    """Gates far below 0, whose sigmoid is a subnormal float32: e^gate is off
    by one of the smallest steps, 2^-149 (its product with the gate by a 70th of
    that), and the value by the 10 U of any gated one."""
    rng = np.random.default_rng(2)
    rows, cols = 150, 260
    gate = rng.uniform(-101, -70, (rows, cols)).astype(np.float32)
    gate[:, 128:256] = rng.uniform(-101, -89, (rows, 128))
    up = (rng.normal(0, 1, (rows, cols)) * 2.0 ** 100).astype(np.float32)
    x = torch.from_numpy(np.concatenate([gate, up], 1))
    e = np.exp(gate.astype(np.float64))
    v = gate * e / (1 + e) * up
    off = np.abs(v) * (10 * H.U + 1.02 * 2.0 ** -149 / e)
    v, off = (v.T, off.T) if transpose else (v, off)
    q, s = run_quantise(x.cuda(), "f32", rows, cols, gated=True, block_rows=block_rows, transpose=transpose)
    M, K = v.shape
    for r in range(s.shape[0]):
        for b in range(s.shape[1]):
            at = (slice(r * block_rows, (r + 1) * block_rows), slice(b * 128, (b + 1) * 128))
            want = np.abs(v[at]).max() / 448
            assert abs(s[r, b] - want) <= off[at].max() / 448 + want * H.U, (r, b, s[r, b], want)
    sc = H.spread(s, block_rows, M, K)
    room = np.maximum(np.abs(v) * 2.0 ** -4, sc * 2.0 ** -10) * (1 + 2.0 ** -10) + 2 * off
    assert (np.abs(H.mxfp8.e4m3_decode(q) * sc - v) <= room).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantise_gated_in_square_blocks_and_batches(dtype, transpose):
    g = torch.Generator().manual_seed(4)
    n, rows, cols = 3, 200, 150
    x = (torch.randn(n, rows, 2 * cols, generator=g) * 3).to(DT[dtype])
    orows, ocols = (cols, rows) if transpose else (rows, cols)
    q = torch.zeros(n, orows, ocols, dtype=torch.uint8, device="cuda")
    s = torch.zeros(n, 2, 2, device="cuda")
    B.reshard_fp8_quantise(B.Fp8Quant(dtype, rows, cols, batch=n, gated=True, block_rows=128, transpose=transpose), ptr(x.cuda()),
                           None, ptr(q), ptr(s), stream())
    for i in range(n):
        gate, up = f64(x[i, :, :cols]), f64(x[i, :, cols:])
        v = gate / (1 + np.exp(-gate)) * up
        v = v.T if transpose else v
        for r in range(2):
            for b in range(2):
                want = np.abs(v[r * 128:(r + 1) * 128, b * 128:(b + 1) * 128]).max() / 448
                assert abs(float(s[i, r, b]) - want) <= want * 11 * H.U
        sc = H.spread(s[i].cpu().numpy(), 128, orows, ocols)
        room = np.maximum(np.abs(v) * 2.0 ** -4, sc * 2.0 ** -10) * (1 + 2.0 ** -10) + np.abs(v) * 16 * H.U
        assert (np.abs(H.mxfp8.e4m3_decode(q[i].cpu().numpy()) * sc - v) <= room).all()


# Streamed rows (few a group), tiles of 64 rows and of 128.
@pytest.mark.parametrize("M,N,K,G", [(40, 64, 128, 16), (40, 64, 128, 3), (1500, 3000, 256, 3)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_matmul_rows_without_a_group_are_left(M, N, K, G, out):
    """Rows before the first offset and behind the last, offsets beyond m
    (cut to it) and below 0, descending ones (an empty group): what a group
    holds is its product, every other row keeps what it had."""
    rng = np.random.default_rng(M)
    a, b = Operand(rng, 1, M, K, 1), Operand(rng, G, N, K, 128)
    at = lambda *p: [int(v * M) for v in p]
    for ends in (at(0, .7, 1.2, 2.2), at(.12, .25, .25, .5), at(0, .75, .5, .62), at(-.2, .1, .1, .1), at(1.5, 1.6, 1.7, 1.8),
                 at(.5, .5, .5, .5), at(.9, .2, .3, 1)):
        off = np.array([ends[0]] * (G - 3) + ends, dtype=np.int32)
        c = Guarded(M, N, DT[out])
        before = c.t.clone()
        mm = B.Fp8Matmul(M, N, K, out, groups=G, a_stride=a.ld, b_stride=b.ld)
        B.reshard_fp8_matmul(mm, ptr(a.dev), ptr(a.sdev), None, ptr(b.dev), ptr(b.sdev), ptr(torch.from_numpy(off).cuda()),
                             c.ptr, stream())
        torch.cuda.synchronize()
        cut = np.clip(off, 0, M)
        held = np.zeros(M, dtype=int)   # groups that name a row: two where offsets descend
        for g in range(G):
            held[cut[g]:max(cut[g], cut[g + 1])] += 1
        for g in range(G):
            rows = [i for i in range(cut[g], max(cut[g], cut[g + 1])) if held[i] == 1]
            want, tol = H.product(a.values[0][rows], b.values[g], -(-K // 128), out)
            H.close(f64(c.t)[rows], want, tol, out, "group %d" % g)
        left = torch.from_numpy(held == 0).cuda()
        assert torch.equal(c.t[left].contiguous().view(torch.uint8), before[left].contiguous().view(torch.uint8))
        assert c.intact()


def outlier_codes(rng, R, K, large, small):
    """Rows whose every eighth column holds `large`, the others `small` (E4M3 codes)."""
    q = np.full((R, K), small, dtype=np.uint8)
    q[:, ::8] = large
    return q


@pytest.mark.parametrize("M,N,K", [(1, 64, 1024), (20, 100, 1040), (40, 200, 1024), (300, 300, 1000), (2900, 3000, 392)])
@pytest.mark.parametrize("b_rows", [128, 1])
def test_matmul_f16_keeps_small_products_next_to_large_ones(M, N, K, b_rows):
    """Large products that cancel: the small ones between them are the result,
    and float32 sums hold them (448 * 448 + 2 * 2 takes 17 bits)."""
    rng = np.random.default_rng(0)
    a, b = Operand(rng, 1, M, K, 1), Operand(rng, 1, N, K, b_rows)
    top, two = 0x7E, 0x40   # 448 and 2
    qa, qb = outlier_codes(rng, M, K, top, two), outlier_codes(rng, N, K, top, two)
    qb[:, 8::16] |= 0x80    # every other large product is negative
    for o, q in ((a, qa), (b, qb)):
        o.dev[0, :, :K] = torch.from_numpy(q).cuda()
        o.sdev.fill_(0.5)
    want, tol = H.product(H.mxfp8.e4m3_decode(qa) * 0.5, H.mxfp8.e4m3_decode(qb) * 0.5, -(-K // 128), "f32")
    c = Guarded(M, N, torch.float16)
    mm = B.Fp8Matmul(M, N, K, "f16", a_stride=a.ld, b_stride=b.ld, b_block_rows=b_rows)
    B.reshard_fp8_matmul(mm, ptr(a.dev), ptr(a.sdev), None, ptr(b.dev), ptr(b.sdev), None, c.ptr, stream())
    torch.cuda.synchronize()
    H.close(f64(c.t), want, tol, "f16", "c")
    assert c.intact()


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M", [3, 40, 700])
def test_matmul_outlier_columns(M, out):
    """Activations with a column in 128 a hundred times the others."""
    rng = np.random.default_rng(M)
    N, K = 300, 1024
    x, w = rng.normal(0, 1, (M, K)), rng.normal(0, 0.02, (N, K))
    x[:, 5::128] *= 100
    (qa, sa), (qb, sb) = H.quantise(x, 1), H.quantise(w, 128)
    want, tol = H.product(H.values(qa, sa, 1), H.values(qb, sb, 128), 8, "f32" if out == "f16" else out)
    c = Guarded(M, N, DT[out])
    B.reshard_fp8_matmul(B.Fp8Matmul(M, N, K, out), ptr(torch.from_numpy(qa).cuda()), ptr(torch.from_numpy(sa).cuda()), None,
                         ptr(torch.from_numpy(qb).cuda()), ptr(torch.from_numpy(sb).cuda()), None, c.ptr, stream())
    torch.cuda.synchronize()
    H.close(f64(c.t), want, tol, out, "c")


@pytest.mark.parametrize("M,N,K", [(2900, 3000, 392), (1900, 3000, 392), (1000, 3000, 4000)])
def test_matmul_f16_many_tiles(M, N, K):
    check_matmul(M, N, K, "f16", c_pad=5, seed=M, factor=2.0 ** -12)
    check_matmul(0, N, K, "f16", groups=[M // 2, 0, 1, M // 3, 65], index_rows=300, tail=9, seed=K, factor=2.0 ** -12)


@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", range(len(matmul_shapes.CASES)))
def test_matmul_every_kernel(case, out, b_rows):
    """Each kernel's forms: plain and gathered rows, every result, both scale forms."""
    _, groups, M, N, K = matmul_shapes.CASES[case]
    factor = 2.0 ** -12 if out == "f16" else 1.0   # f16 results that do not overflow
    check_matmul(M, N, K, out, groups=groups, b_rows=b_rows, c_pad=3, seed=case, factor=factor)
    check_matmul(M, N, K, out, groups=groups, b_rows=b_rows, index_rows=300, seed=case, factor=factor)
