"""GPU tests of the operators around the recurrence against their fp64 / integer oracle.

Tolerances, from the arithmetic (e = torch.finfo(t).eps / 2 is half a step of the type t):
  norm_quant  the residual's sum is rounded to fp32 and then to t: (e + 2^-23) |h|. The sum of squares
              of a row is at most 64 additions per thread and 40 across threads, each off by
              2^-24 of the sum, and rsqrt, two products and the division by 448 add a few
              steps: y, the scale and y / s are within R = 128 * 2^-24 relative. q rounds y / s (half a step: 2^-4
              relative, or 2^-10 among the subnormals).
  fp8_matmul  products are exact in fp32; at most 128 additions within a group, one per group and
              the scales' product, each off by at most a step (2^-23, a truncating adder) of the sum of the
              magnitudes S: (132 + K / 128) 2^-23 S, and e of the result.
  batch_maps  integers: equal.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import layer_ops as lo

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available()
    from linear_attention_state_recurrent_gb300 import build
    build.build()
    from linear_attention_state_recurrent_gb300 import kda as k
    return k


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.to(torch.float64).cpu().numpy()


def rand(rows, cols, dtype, seed, scale=1.0, pad=0):
    """[rows, cols] normal values in a buffer whose rows are `pad` elements longer (NaN there)."""
    g = torch.Generator().manual_seed(seed)
    t = torch.full((rows, cols + pad), math.nan, dtype=dtype, device="cuda")
    t[:, :cols] = (torch.randn(rows, cols, generator=g) * scale).to(dtype).cuda()
    return t[:, :cols]


# ---- kda_norm_quant -----------------------------------------------------------------------


def check_norm(kda, x, weight, eps=1e-5, residual=None, want_y=False, **out):
    rows, cols = x.shape
    xs, rs = f64(x), None if residual is None else f64(residual)
    y = torch.empty_like(x) if want_y else out.pop("y", None)
    q, s, ro = kda.kda_norm_quant(x, weight, eps, residual=residual, y=y, **out)
    torch.cuda.synchronize()
    h, ey, es, ev = lo.norm_quant(xs, rs, None if weight is None else f64(weight), eps)
    R = 128 * 2.0 ** -24
    if residual is None:
        assert ro is None
    else:
        assert np.all(np.abs(f64(ro) - h) <= (half_step(x.dtype) + 2.0 ** -23) * np.abs(h))
    if y is not None:
        e = half_step(x.dtype)
        small = torch.finfo(x.dtype).smallest_normal * 2 * e    # half a subnormal step of the type
        assert np.all(np.abs(f64(y) - ey) <= (e + R) * np.abs(ey) + small)
    assert np.all(np.abs(f64(s) - es) <= R * es)
    # y / s is off by R relative before it is rounded; a value pushed over a border of the rounding
    # lands on the neighbour, so the bound is half a step of the larger of the two
    assert np.all(np.abs(f64(q) - ev) <= np.maximum(2.0 ** -4 * np.abs(ev), 2.0 ** -10) * (1 + 2.0 ** -10) + R * np.abs(ev))
    top = np.stack([np.abs(f64(q))[:, g:g + 128].max(1) for g in range(0, cols, 128)], 1)
    assert np.all((top == 448) | (es <= 2.0 ** -126 * (1 + 2.0 ** -10)))


@pytest.mark.parametrize("cols", [1, 8, 127, 128, 129, 256, 1000, 1024, 1032, 4096, 4104, 5003, 16384])
@pytest.mark.parametrize("rows", [1, 3, 600])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_norm_quant_sizes(kda, rows, cols, dtype):
    x, r = rand(rows, cols, dtype, 1, 2.0), rand(rows, cols, dtype, 2)
    w = 1 + 0.2 * rand(1, cols, FP32, 3)[0]
    check_norm(kda, x, w, residual=r, want_y=True)
    check_norm(kda, x, None)


@pytest.mark.parametrize("cols", [16385, 16392, 20000, 32761, 32768])
def test_norm_quant_wide_rows(kda, cols):
    for dtype, pad in ((BF16, 0), (FP32, 3)):
        x = rand(2, cols, dtype, 4, pad=pad)
        check_norm(kda, x, torch.ones(cols, device="cuda"), residual=rand(2, cols, dtype, 5), want_y=True)


@pytest.mark.parametrize("pad,offset", [(8, 0), (5, 0), (8, 8), (8, 1), (3, 5)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_norm_quant_strides_and_offsets(kda, dtype, pad, offset):
    rows, cols = 5, 392
    def view(t):
        buf = torch.full((rows * (cols + pad) + offset + 16,), math.nan, dtype=t.dtype, device="cuda") if t.dtype != E4M3 else \
            torch.full((rows * (cols + pad) + offset + 16,), 7.0, device="cuda").to(E4M3)
        v = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        v.copy_(t)
        return buf, v
    x, r = view(rand(rows, cols, dtype, 6))[1], view(rand(rows, cols, dtype, 7))[1]
    bufs = {"residual_out": view(torch.zeros(rows, cols, dtype=dtype, device="cuda")), "y": view(torch.zeros(rows, cols, dtype=dtype, device="cuda")),
            "q": view(torch.zeros(rows, cols, device="cuda").to(E4M3))}
    before = {k: b.clone() for k, (b, _) in bufs.items()}
    scales = torch.full((rows, 9), 5.0, device="cuda")[:, 1:9:2]   # 4 groups, a stride of 2
    check_norm(kda, x, rand(1, cols + offset, FP32, 8)[0, offset:], residual=r, scales=scales, **{k: v for k, (_, v) in bufs.items()})
    for k, (b, v) in bufs.items():   # nothing outside the rows was written
        v.copy_(torch.zeros(rows, cols, device="cuda"))
        old = before[k]
        old[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols].copy_(torch.zeros(rows, cols, device="cuda"))
        assert torch.equal(b.view(torch.uint8), old.view(torch.uint8))
    assert torch.equal(scales._base[:, ::2], torch.full((rows, 5), 5.0, device="cuda"))


@pytest.mark.parametrize("weight", [True, False])
def test_norm_quant_in_place_residual(kda, weight):
    x, r = rand(9, 640, BF16, 9), rand(9, 640, BF16, 10)
    w = torch.ones(640, device="cuda") if weight else None
    q0, s0, ro0 = kda.kda_norm_quant(x, w, residual=r)
    q1, s1, ro1 = kda.kda_norm_quant(x, w, residual=r, residual_out=r, y=x)
    assert ro1 is r and torch.equal(ro0, ro1) and torch.equal(s0, s1) and torch.equal(q0.view(torch.uint8), q1.view(torch.uint8))
    # y is q * s up to half a step of e4m3
    assert torch.all((x.float() - q1.float() * s1.repeat_interleave(128, 1)).abs() <= 2.0 ** -4 * x.float().abs() + 2.0 ** -9 * s1.max() + 2.0 ** -7 * x.float().abs())


def test_norm_quant_zeros_and_tiny_values(kda):
    x = torch.zeros(4, 256, device="cuda")
    x[1] = 2.0 ** -140
    x[2, 3] = -1e-30
    q, s, _ = kda.kda_norm_quant(x)
    assert torch.all(s[0] == 2.0 ** -126) and torch.all(q.float()[[0, 3]] == 0) and not s.isnan().any()
    assert torch.all(s[1] == 2.0 ** -126) and q.float()[2, 3] == -448
    q, s, _ = kda.kda_norm_quant(x, torch.ones(256, device="cuda"), 0.0)   # eps 0 and a zero row: 0 / 0
    assert q.float()[0].isnan().all() and s[0].isnan().all()
    assert not kda.kda_norm_quant(x, torch.ones(256, device="cuda"), 1e-6)[0].float().isnan().any()


def test_norm_quant_nan_and_inf(kda):
    x = rand(6, 384, FP32, 11)
    x[1, 130], x[2, 5], x[3, 383] = math.nan, math.inf, -math.inf
    q, s, _ = kda.kda_norm_quant(x)
    qf = q.float()
    assert s[1].isnan().tolist() == [False, True, False] and qf[1, 128:256].isnan().all() and not qf[1, :128].isnan().any()
    assert s[2, 0] == math.inf and qf[2, 5].isnan() and torch.all(qf[2, :5] == 0) and s[3, 2] == math.inf and qf[3, 383].isnan()
    clean = kda.kda_norm_quant(x[4:])
    assert torch.equal(qf[4:], clean[0].float()) and torch.equal(s[4:], clean[1])
    q, s, _ = kda.kda_norm_quant(x, torch.ones(384, device="cuda"))
    qf = q.float()
    assert qf[1].isnan().all() and s[1].isnan().all()
    assert qf[2, :128].isnan().all() and torch.all(qf[2, 128:] == 0) and not qf[[0, 4, 5]].isnan().any()


def test_norm_quant_of_no_rows(kda):
    q, s, _ = kda.kda_norm_quant(torch.empty(0, 256, dtype=BF16, device="cuda"), torch.ones(256, device="cuda"))
    assert q.shape == (0, 256) and s.shape == (0, 2)


# ---- kda_fp8_matmul -----------------------------------------------------------------------


def operands(M, N, K, seed, pad=(0, 0), group_major=True):
    """e4m3 a [M, K] and w [N, K] with every magnitude of the type, rows `pad` bytes longer than needed
    (NaN bytes there) and scales over a wide range."""
    g = torch.Generator().manual_seed(seed)
    def codes(rows, extra):
        c = torch.randint(0, 256, (rows, K), generator=g, dtype=torch.uint8)
        c = torch.where((c & 0x7F) == 0x7F, c & 0x80, c)          # no NaN
        buf = torch.full((rows, K + extra), 0x7F, dtype=torch.uint8)
        buf[:, :K] = c
        return buf.cuda().view(E4M3)[:, :K]
    G = -(-K // 128)
    a, w = codes(M, pad[0]), codes(N, pad[1])
    sa = torch.exp(torch.randn(M, G, generator=g)).cuda()
    sw = torch.exp(torch.randn(-(-N // 128), G, generator=g)).cuda()
    return a, sa.t().contiguous().t() if group_major else sa, w, sw


def check_matmul(kda, a, sa, w, sw, dtype=BF16, out=None):
    M, K = a.shape
    N = w.shape[0]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = kda.kda_fp8_matmul(a, sa, w, sw, out=out, out_dtype=dtype, err_flags=err)
    torch.cuda.synchronize()
    ref, mag = lo.fp8_matmul(f64(a), f64(sa), f64(w), f64(sw))
    assert err.item() == 0 and out.shape == (M, N)
    got = f64(out)
    tol = (132 + K / 128) * 2.0 ** -23 * mag + half_step(out.dtype) * np.abs(ref)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5])
    return out


def up16(n):
    return -n % 16


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 33, 64, 65, 100, 128, 129, 200, 256, 257])
@pytest.mark.parametrize("N,K", [(32, 128), (128, 256), (129, 512), (1111, 1301), (640, 4096)])
def test_fp8_matmul_sizes(kda, M, N, K):
    a, sa, w, sw = operands(M, N, K, M + N + K, (up16(K), up16(K)))
    check_matmul(kda, a, sa, w, sw)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 7, 16), (5, 130, 15), (3, 128, 127), (130, 3, 129), (64, 64, 17), (300, 300, 300),
                                   (1, 20512, 64), (2050, 33, 640), (1000, 1000, 144)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_fp8_matmul_odd_sizes_and_types(kda, M, N, K, dtype):
    a, sa, w, sw = operands(M, N, K, M + 3 * N + K, (up16(K), up16(K)))
    check_matmul(kda, a, sa, w, sw, dtype)


def test_fp8_matmul_fp16_out(kda):
    a, sa, w, sw = operands(70, 200, 384, 5)
    check_matmul(kda, a, sa * 1e-4, w, sw * 1e-2, FP16)


@pytest.mark.parametrize("M", [3, 150])
@pytest.mark.parametrize("pad", [(1, 0), (0, 5), (3, 3), (16, 32)])
def test_fp8_matmul_row_strides(kda, M, pad):
    a, sa, w, sw = operands(M, 140, 272, 6, pad)
    check_matmul(kda, a, sa, w, sw)


@pytest.mark.parametrize("M", [3, 150])
def test_fp8_matmul_unaligned_bases_and_views(kda, M):
    a, sa, w, sw = operands(M + 1, 301, 400, 7)
    fa, fw = a.reshape(-1), w.reshape(-1)
    check_matmul(kda, fa[1:1 + M * 400].view(M, 400), sa[1:], fw[16:16 + 300 * 400].view(300, 400), sw)
    check_matmul(kda, a[:M:2], sa[:M:2], w[1::3], sw[:1], FP32)          # every other row, contiguous scales no longer
    buf = torch.full((M, 320), 9.0, dtype=FP32, device="cuda")
    check_matmul(kda, a[:M], sa[:M].contiguous(), w, sw.t().contiguous().t(), out=buf[:, 3:304])
    assert torch.all(buf[:, :3] == 9) and torch.all(buf[:, 304:] == 9)


ARRANGEMENTS = [(24, 300, 640), (60, 500, 300), (60, 9000, 140), (100, 300, 640), (300, 1500, 300), (700, 4200, 140), (1500, 600, 260)]


@pytest.mark.parametrize("M,N,K", ARRANGEMENTS)
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("aligned", [True, False])
def test_fp8_matmul_every_arrangement(kda, M, N, K, dtype, aligned):
    """Each way a call may be cut up, with outputs on and off 16-byte boundaries and scales in either order."""
    a, sa, w, sw = operands(M, N, K, M, (up16(K), up16(K)), group_major=aligned)
    edge = 16 if aligned else 5
    buf = torch.full((M, N + 2 * edge + up16(N) * aligned), 9.0, dtype=dtype, device="cuda")
    check_matmul(kda, a, sa, w, sw, out=buf[:, edge:edge + N])
    assert torch.all(buf[:, :edge] == 9) and torch.all(buf[:, edge + N:] == 9)


@pytest.mark.parametrize("M,N,K", ARRANGEMENTS)
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_fp8_matmul_rounds_the_fp32_result_once(kda, M, N, K, dtype):
    """How a call is cut up does not depend on the output's type, so a 16-bit output is the fp32 one, rounded."""
    a, sa, w, sw = operands(M, N, K, M, (up16(K), up16(K)))
    sa, sw = sa * 1e-4, sw * 1e-2
    full = kda.kda_fp8_matmul(a, sa, w, sw, out_dtype=FP32)
    assert torch.equal(kda.kda_fp8_matmul(a, sa, w, sw, out_dtype=dtype), full.to(dtype))


@pytest.mark.parametrize("M,N,K", [(1025, 16, 16), (1311, 167, 365), (1101, 207, 725), (1968, 600, 684), (1100, 40, 4000),
                                   (9038, 243, 168), (16809, 37, 479), (2500, 1500, 1040)])
@pytest.mark.parametrize("aligned", [True, False])
def test_fp8_matmul_many_rows_of_few_columns(kda, M, N, K, aligned):
    """More rows than one wave of narrow tiles, where both the narrow and the wide arrangement are open."""
    a, sa, w, sw = operands(M, N, K, M, (up16(K), up16(K)), group_major=aligned)
    edge = 16 if aligned else 5
    buf = torch.full((M, N + 2 * edge + up16(N) * aligned), 9.0, dtype=BF16, device="cuda")
    check_matmul(kda, a, sa, w, sw, out=buf[:, edge:edge + N])
    assert torch.all(buf[:, :edge] == 9) and torch.all(buf[:, edge + N:] == 9)


@pytest.mark.parametrize("M", [65535 * 128, 65535 * 128 + 1])
def test_fp8_matmul_rows_past_a_grid_axis(kda, M):
    """Rows of ones count their columns: exact, whichever side of the grid's limit the rows end on."""
    a = torch.ones(M, 16, device="cuda").to(E4M3)
    w = torch.ones(3, 16, device="cuda").to(E4M3)
    w.view(torch.uint8)[1] = 0
    sa = torch.arange(M, device="cuda").remainder(5).add(1).to(FP32)[:, None]
    sw = torch.full((1, 1), 0.5, device="cuda")
    out = kda.kda_fp8_matmul(a, sa, w, sw)
    assert torch.equal(out, torch.tensor([8.0, 0.0, 8.0], device="cuda") * sa)


@pytest.mark.parametrize("M,N,K", [(2500, 1500, 1040), (1300, 1, 40), (1300, 3, 128), (1300, 7, 16), (1500, 263, 300), (1100, 4097, 140)])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_fp8_matmul_leaves_the_columns_beside_it(kda, M, N, K, dtype):
    """A view into wider rows, on 16-byte boundaries, that ends inside 16 bytes."""
    a, sa, w, sw = operands(M, N, K, M, (up16(K), up16(K)))
    buf = torch.full((M, N + 32 + up16(N)), 9.0, dtype=dtype, device="cuda")
    if dtype == FP16:                                             # the range of its normal numbers, near enough
        sa, sw = sa * 1e-3, sw * 1e-3
        out = kda.kda_fp8_matmul(a, sa, w, sw, out=buf[:, 16:16 + N])
        assert torch.equal(out, kda.kda_fp8_matmul(a, sa, w, sw, out_dtype=FP32).to(FP16))
    else:
        check_matmul(kda, a, sa, w, sw, out=buf[:, 16:16 + N])
    assert torch.all(buf[:, :16] == 9) and torch.all(buf[:, 16 + N:] == 9)


def test_fp8_matmul_split_of_a_long_inner_axis(kda):
    for M in (1, 20, 130):
        a, sa, w, sw = operands(M, 40, 16384 + 48, 8)
        check_matmul(kda, a, sa, w, sw, FP32)


def test_fp8_matmul_nan_stays_in_its_row_and_column(kda):
    for M in (5, 140):
        a, sa, w, sw = operands(M, 150, 256, 9)
        clean = kda.kda_fp8_matmul(a, sa, w, sw)
        a.view(torch.uint8)[2, 200] = 0x7F
        w.view(torch.uint8)[149, 0] = 0xFF
        out = kda.kda_fp8_matmul(a, sa, w, sw)
        assert out[2].isnan().all() and out[:, 149].isnan().all()
        keep = torch.ones(M, 150, dtype=torch.bool, device="cuda")
        keep[2], keep[:, 149] = False, False
        assert torch.equal(out[keep], clean[keep])


def test_fp8_matmul_empty(kda):
    a, sa, w, sw = operands(4, 12, 128, 10)
    assert kda.kda_fp8_matmul(a[:0], sa[:0], w, sw).shape == (0, 12)
    assert kda.kda_fp8_matmul(a, sa, w[:0], sw[:0]).shape == (4, 0)
    out = kda.kda_fp8_matmul(a[:, :0], sa[:, :0], w[:, :0], sw[:, :0])
    assert out.shape == (4, 12) and not out.any()


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (128, 4096, 2048), (777, 1024, 2048)])
def test_fp8_matmul_repeats_bit_for_bit(kda, M, N, K):
    a, sa, w, sw = operands(M, N, K, 11)
    first = kda.kda_fp8_matmul(a, sa, w, sw, out_dtype=FP32)
    for _ in range(5):
        assert torch.equal(first, kda.kda_fp8_matmul(a, sa, w, sw, out_dtype=FP32))


@pytest.mark.parametrize("M,N,K", [(33494, 512, 256), (20, 20512, 1024), (4200, 4100, 520)])
def test_fp8_matmul_many_tiles(kda, M, N, K):
    """Sizes past one wave, checked on sampled rows and columns."""
    a, sa, w, sw = operands(M, N, K, 12, (up16(K), up16(K)))
    out = kda.kda_fp8_matmul(a, sa, w, sw, out_dtype=FP32)
    g = torch.Generator().manual_seed(1)
    rows = torch.cat([torch.randint(0, M, (200,), generator=g), torch.tensor([0, M - 1])]).cuda()
    ref, mag = lo.fp8_matmul(f64(a.view(torch.uint8)[rows].view(E4M3)), f64(sa[rows]), f64(w), f64(sw))
    tol = (132 + K / 128) * 2.0 ** -23 * mag + half_step(FP32) * np.abs(ref)
    assert np.all(np.abs(f64(out[rows]) - ref) <= tol)
    assert not out.isnan().any()


# ---- kda_batch_maps -----------------------------------------------------------------------


def maps_case(seed, R, page, width, num_tokens, lens, context, num_free=None, state_stride=1, extra_rows=0):
    r = np.random.default_rng(seed)
    q = np.asarray([lens(r) for _ in range(R)], np.int64)
    c = np.asarray([context(r) for _ in range(R)], np.int64)
    pages = r.permutation(R * width + 70).astype(np.int32)
    table = np.full((R, width), -1, np.int32)
    for i in range(R):
        have = min(-(-max(int(c[i]), 0) // page), width)
        table[i, :have] = pages[i * width:i * width + have]
    free = pages[R * width:] if num_free is None else r.permutation(R * width + 70 + num_free)[:num_free].astype(np.int32)
    slots = r.permutation(R * state_stride + 5).astype(np.int32)[:R * state_stride].reshape(R, state_stride)
    return dict(q=q, c=c, table=table, free=free, slots=slots, page=page, num_pages=int(max(pages.max(), free.max() if len(free) else 0)) + 1,
                num_tokens=num_tokens)


def check_maps(kda, m, free_count=None, stream=None):
    def up(a):
        return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    free_count = len(m["free"]) if free_count is None else free_count
    want, want_err = lo.batch_maps(m["q"], m["c"], m["slots"][:, 0], m["table"], m["free"], free_count, m["page"], m["num_pages"],
                                   m["num_tokens"])
    R, width = m["table"].shape
    table = torch.full((R, width + 3), -7, dtype=torch.int32, device="cuda")[:, :width]
    table.copy_(up(m["table"]))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    count = up([free_count])
    args = (up(m["q"]), up(m["c"]), up(m["slots"])[:, 0], table, up(m["free"]), count, m["page"])
    for _ in range(2):   # the inputs do not change, so a repeat writes the same
        got = kda.kda_batch_maps(*args, num_pages=m["num_pages"], num_tokens=m["num_tokens"], err_flags=err, stream=stream)
    torch.cuda.synchronize()
    for name, t in got._asdict().items():
        np.testing.assert_array_equal(t.cpu().numpy(), want[name], err_msg=name)
    np.testing.assert_array_equal(table.cpu().numpy(), want["block_table"])
    assert torch.all(table._base[:, width:] == -7) and count.item() == free_count
    assert err.item() == want_err


@pytest.mark.parametrize("R", [1, 2, 31, 32, 33, 127, 128, 1000, 4097, 9001])
def test_batch_maps_decodes(kda, R):
    check_maps(kda, maps_case(R, R, 16, 5, R + 3, lambda r: 1, lambda r: int(r.integers(0, 79)), num_free=R + 1))


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("R", [1, 5, 100, 4500])
def test_batch_maps_mixed_lengths(kda, R, page):
    m = maps_case(R + page, R, page, -(-140 // page), 0, lambda r: int(r.choice([0, 1, 1, 2, 17, 40])),
                  lambda r: int(r.choice([0, 1, page, 5 * page - 1, 99])) % 100, num_free=50 * R + 50, state_stride=3)
    m["num_tokens"] = int(m["q"].sum()) + 5
    check_maps(kda, m)


def test_batch_maps_long_prefills_across_ctas(kda):
    m = maps_case(3, 4, 64, 520, 0, lambda r: int(r.integers(5000, 20000)), lambda r: int(r.integers(0, 10000)), num_free=2000)
    m["num_tokens"] = int(m["q"].sum())
    check_maps(kda, m)


def test_batch_maps_no_requests_no_tokens(kda):
    check_maps(kda, maps_case(4, 0, 16, 4, 7, None, None, num_free=3))
    check_maps(kda, maps_case(5, 3, 16, 4, 0, lambda r: 0, lambda r: 5, num_free=3))
    check_maps(kda, maps_case(5, 3, 16, 4, 9, lambda r: 0, lambda r: 5, num_free=0))


@pytest.mark.parametrize("num_tokens", [0, 1, 50, 51, 149])
def test_batch_maps_cuts_off_at_the_capacity(kda, num_tokens):
    m = maps_case(6, 40, 8, 8, num_tokens, lambda r: int(r.choice([1, 3, 9])), lambda r: int(r.integers(0, 30)), num_free=400)
    assert m["q"].sum() > num_tokens
    check_maps(kda, m)


@pytest.mark.parametrize("free_count", [0, 1, 13, -5, 10 ** 6])
def test_batch_maps_runs_out_of_pages(kda, free_count):
    m = maps_case(7, 30, 8, 8, 0, lambda r: int(r.choice([1, 3, 9])), lambda r: int(r.integers(0, 30)), num_free=20)
    m["num_tokens"] = int(m["q"].sum())
    check_maps(kda, m, free_count)


def test_batch_maps_full_rows_and_bad_pages(kda):
    m = maps_case(8, 20, 8, 3, 0, lambda r: int(r.choice([1, 3, 9])), lambda r: int(r.integers(0, 60)), num_free=60)
    m["table"][3, 0], m["table"][5, 1] = m["num_pages"], -4
    m["free"][-1] = m["num_pages"] + 1
    m["num_tokens"] = int(m["q"].sum())
    check_maps(kda, m)


def test_batch_maps_bad_lengths(kda):
    m = maps_case(9, 50, 16, 6, 200, lambda r: int(r.choice([0, 1, 2, 5])), lambda r: int(r.integers(0, 60)), num_free=100)
    m["q"][4], m["c"][7], m["q"][11], m["c"][11] = -1, -3, 2 ** 31 - 1, 1
    check_maps(kda, m)
    m["q"][20] = 2 ** 31 - 1 - 100 - m["c"][20]   # in range, cut off at the capacity
    check_maps(kda, m)


def test_batch_maps_slots_past_32_bits(kda):
    m = maps_case(10, 6, 2 ** 20, 2, 0, lambda r: int(r.integers(1, 9)), lambda r: 2 ** 20 - 3, num_free=12)
    m["free"] += 10000
    m["num_pages"] += 10000
    m["num_tokens"] = int(m["q"].sum())
    check_maps(kda, m)


# ---- streams and graphs -------------------------------------------------------------------


def step(kda, x, w, a8, sa, wq, sw, maps):
    q, s, _ = kda.kda_norm_quant(x, w)
    y = kda.kda_fp8_matmul(q, s, wq, sw)
    return y, kda.kda_batch_maps(*maps, 16, num_pages=64, num_tokens=40)


def step_inputs():
    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    x, w = rand(20, 512, BF16, 20), torch.ones(512, device="cuda")
    a, sa, wq, sw = operands(20, 260, 512, 21)
    return x, w, a, sa, wq, sw, (i32([1, 20, 3]), i32([5, 0, 30]), i32([4, 5, 6]), i32([[0, -1, -1], [-1, -1, -1], [1, 2, -1]]),
                                 i32([10, 11, 12, 13]), i32([4]))


def test_on_a_side_stream(kda):
    inp = step_inputs()
    want = step(kda, *inp)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step(kda, *inp)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and all(torch.equal(a, b) for a, b in zip(want[1], got[1]))


def test_in_a_graph(kda):
    inp = step_inputs()
    want = step(kda, *inp)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(kda, *inp)
    inp[0].mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(-want[0], got[0]) and all(torch.equal(a, b) for a, b in zip(want[1], got[1]))


def test_first_calls_inside_a_capture():
    """What a first call on a device looks up and sets is allowed while a stream is captured."""
    code = """
import sys; sys.path.insert(0, %r)
import torch
from linear_attention_state_recurrent_gb300 import kda
x = torch.randn(300, 512, device="cuda").to(torch.bfloat16)
w = torch.ones(256, 512, device="cuda").to(torch.float8_e4m3fn)
sw = torch.ones(2, 4, device="cuda")
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
args = (i32(1, 2), i32(0, 3), i32(4, 5), torch.zeros(2, 4, dtype=torch.int32, device="cuda"), i32(7, 8), i32(2), 16)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    q, s, _ = kda.kda_norm_quant(x)
    y = [kda.kda_fp8_matmul(q[:m], s[:m], w, sw) for m in (1, 20, 50, 100, 300)]
    m = kda.kda_batch_maps(*args, num_pages=16, num_tokens=4)
g.replay()
torch.cuda.synchronize()
assert all(torch.isfinite(t.float()).all() for t in y) and m.cu_seqlens.tolist() == [0, 1, 3]
print("captured")
""" % os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
