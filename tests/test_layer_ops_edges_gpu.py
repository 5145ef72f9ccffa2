"""Edges of the operators around the recurrence where a result could be right nearly everywhere: values between
two of a type's, streams other than the current one, waits that give up, and every way a product is cut up."""
import numpy as np
import pytest
import torch

from tests.test_layer_ops_gpu import check_matmul, operands, up16

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


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def weights(n, k, seed):
    """e4m3 [n, k] with scales."""
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, k, generator=g).to(E4M3).cuda(), torch.exp(torch.randn(-(-n // 128), -(-k // 128), generator=g)).cuda()


# ---- kda_norm_quant: values between two of e4m3 -------------------------------------------


def midpoints():
    """Every value half way between two neighbours of e4m3, as fp64."""
    subnormal = [(m + 0.5) * 2.0 ** -9 for m in range(8)]
    normal = [(8 + m + 0.5) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)]
    return np.array([v for v in subnormal + normal if v < 448])


def tie_rows(dtype):
    """Rows of one group whose largest value gives a scale of j / 64 exactly, the others midpoints of e4m3 times
    that scale where the type holds them (else 0): y / s is the midpoint, with nothing to round."""
    reciprocal = np.float32(1) / np.float32(448)
    rows, want = [], []
    for j in range(1, 2000, 2):
        if np.float32(7 * j) * reciprocal != np.float32(j / 64) or torch.tensor(7.0 * j).to(dtype).double() != 7 * j:
            continue
        for sign in (1, -1):
            for half in np.array_split(midpoints(), 2):
                v = torch.zeros(128, dtype=torch.float64)
                v[1:1 + len(half)] = torch.from_numpy(sign * half)
                x = v * (j / 64)
                held = x.to(dtype).double() == x
                x, v = torch.where(held, x, 0), torch.where(held, v, 0)
                x[0], v[0] = 7 * j, 448
                rows.append(x.to(dtype))
                want.append(v.float())
    return torch.stack(rows), torch.stack(want)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("pad", [0, 1])   # rows on 16-byte boundaries and off them
def test_norm_quant_rounds_midpoints_to_even(kda, dtype, pad):
    x, v = tie_rows(dtype)
    assert (v != 0).sum() > 200
    buf = torch.zeros(x.shape[0], 128 + pad, dtype=dtype, device="cuda")
    buf[:, :128] = x.cuda()
    q, s, _ = kda.kda_norm_quant(buf[:, :128])
    assert torch.equal(s[:, 0].cpu(), (x[:, 0].float() / 448))
    assert torch.equal(q.float().cpu(), v.to(E4M3).float())


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_norm_quant_rounds_the_quotient_by_its_scale(kda, dtype):
    """q is the nearest e4m3 of y / s in fp32, for the scale that is returned: exactly, whatever the values."""
    g = torch.Generator().manual_seed(31)
    x = (torch.randn(2000, 1024, generator=g) * torch.exp(2 * torch.randn(2000, 1, generator=g))).to(dtype).cuda()
    q, s, _ = kda.kda_norm_quant(x)
    quotient = (x.double() / s.double().repeat_interleave(128, 1)).float().clamp(-448, 448)
    assert torch.equal(q.float(), quotient.to(E4M3).float())


# ---- every way a product is cut up ---------------------------------------------------------

# rows of a per tile, whether the inner axis is split, the least and the most rows of w per tile, and a size that gets there
WAYS = {"thin 16": (16, False, 128, 128, (9, 300, 300)), "thin 16 split": (16, True, 128, 128, (9, 300, 1040)),
        "thin 32": (32, False, 128, 128, (24, 300, 300)), "thin 32 split": (32, True, 128, 128, (24, 500, 2100)),
        "thin 64": (64, False, 128, 128, (37, 12374, 529)), "thin 64 split": (64, True, 128, 128, (60, 1500, 1040)),
        "slim, one chunk": (128, False, 16, 64, (100, 300, 300)), "slim, one chunk, split": (128, True, 16, 64, (130, 300, 1040)),
        "slim, two chunks": (128, False, 80, 128, (130, 9000, 140)), "slim, two chunks, split": (128, True, 80, 128, (100, 1500, 2100)),
        "slim, four chunks": (128, False, 144, 256, (700, 4200, 140)), "slim, four chunks, split": (128, True, 144, 256, (300, 1500, 8200)),
        "wide": (256, False, 256, 256, (2500, 1500, 1040)), "wide, few columns": (256, False, 256, 256, (19859, 2, 17)),
        "wide, a warp's columns": (256, False, 256, 256, (21674, 64, 17)), "wide, an edge": (256, False, 256, 256, (9961, 260, 28)),
        "general": (0, False, 64, 64, (70, 130, 261))}


def product(way):
    """The operands of one way, with scales in either order."""
    rows, _, _, _, (M, N, K) = WAYS[way]
    pad = (1, 0) if rows == 0 else (up16(K), up16(K))
    return operands(M, N, K, M + N, pad, group_major=N % 8 == 0)


@pytest.mark.parametrize("way", WAYS)
def test_fp8_matmul_plan(kda, way):
    """The sizes below reach what they are there for: a change of the plans that empties a test fails here."""
    rows, split, least, most, _ = WAYS[way]
    a, _, w, _ = product(way)
    got = kda.kda_fp8_matmul_plan(a, w)
    assert got[0] == rows and (got[1] > 1) == split and least <= got[2] <= most


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("aligned", [True, False])
def test_fp8_matmul_every_way(kda, way, dtype, aligned):
    """Each kernel, split and not, with outputs of each type on and off 16-byte boundaries, in wider rows whose other columns
    stay as they were. A 16-bit output is the fp32 one, rounded once: fp16 is compared with that (its subnormals have
    no relative bound), the others with 64 bits."""
    a, sa, w, sw = product(way)
    M, N = a.shape[0], w.shape[0]
    edge = 16 if aligned else 5
    buf = torch.full((M, N + 2 * edge + up16(N) * aligned), 9.0, dtype=dtype, device="cuda")
    out = buf[:, edge:edge + N]
    if dtype == FP16:
        sa, sw = sa * 1e-4, sw * 1e-2
        kda.kda_fp8_matmul(a, sa, w, sw, out=out)
        assert torch.equal(out, kda.kda_fp8_matmul(a, sa, w, sw, out_dtype=FP32).to(FP16))
    else:
        check_matmul(kda, a, sa, w, sw, out=out)
    assert torch.all(buf[:, :edge] == 9) and torch.all(buf[:, edge + N:] == 9)


@pytest.mark.parametrize("way", [w for w in WAYS if "split" in w] + ["thin 64", "wide", "wide, an edge"])
def test_fp8_matmul_every_way_repeats_bit_for_bit(kda, way):
    a, sa, w, sw = product(way)
    first = kda.kda_fp8_matmul(a, sa, w, sw, out_dtype=FP32)
    for _ in range(20):
        assert torch.equal(first, kda.kda_fp8_matmul(a, sa, w, sw, out_dtype=FP32))


# ---- waits that give up -------------------------------------------------------------------


@pytest.mark.parametrize("M,N,K", [(1, 40, 16432), (20, 40, 16432), (50, 40, 16432), (130, 40, 16432),   # the inner axis split
                                   (9, 20512, 256), (100, 20512, 256), (4000, 1500, 1040)])              # and not
def test_fp8_matmul_whose_waits_give_up_leaves_out_alone(kda, M, N, K):
    """Sums that wait for scales which never come are not stored, neither a CTA's own nor those of a split that
    it is part of; the error word says so, and the next call on the context is right."""
    a, sa = weights(M, K, 51)
    sa = sa.repeat_interleave(128, 0)[:M].contiguous()
    w, sw = weights(N, K, 52)
    err = i32(0)
    want = kda.kda_fp8_matmul(a, sa, w, sw, err_flags=err)
    assert err.item() == 0
    out = torch.full((M, N), 9.0, dtype=BF16, device="cuda")
    kda.kda_selftest_fp8_matmul(a, sa, w, sw, out, err)
    torch.cuda.synchronize()
    assert err.item() == kda.KDA_ERRFLAG_TIMEOUT
    assert torch.all(out == 9)
    err.zero_()
    assert torch.equal(kda.kda_fp8_matmul(a, sa, w, sw, out=out, err_flags=err), want) and err.item() == 0


def test_fp8_matmul_selftest_stalls_nothing_that_is_not_there(kda):
    a, sa = weights(128, 256, 53)
    w, sw = weights(200, 256, 54)
    err, out = i32(0), torch.empty(128, 200, dtype=BF16, device="cuda")
    sa = sa.repeat_interleave(128, 0)
    kda.kda_selftest_fp8_matmul(a, sa, w, sw, out, err, stalled=7)   # two groups: clusters of two at most
    assert torch.equal(out, kda.kda_fp8_matmul(a, sa, w, sw)) and err.item() == 0


# ---- streams other than the current one ---------------------------------------------------


def calls(kda):
    """The calls that allocate, each with outputs of a megabyte or more."""
    g = torch.Generator().manual_seed(41)
    x, r = torch.randn(2, 1500, 2048, generator=g).to(BF16).cuda()
    q, s, _ = kda.kda_norm_quant(x)
    (w, sw), ones = weights(1100, 2048, 42), torch.ones(2048, device="cuda")
    maps = (i32(300000, 1, 200000), i32(0, 7, 3), i32(4, 5, 6), torch.zeros(3, 6000, dtype=torch.int32, device="cuda"),
            torch.arange(9000, dtype=torch.int32, device="cuda"), i32(9000), 100)
    return {"norm_quant": lambda stream: kda.kda_norm_quant(x, ones, residual=r, stream=stream),
            "fp8_matmul": lambda stream: (kda.kda_fp8_matmul(q, s, w, sw, stream=stream),),
            "batch_maps": lambda stream: kda.kda_batch_maps(*maps, num_pages=9000, num_tokens=500001, stream=stream)}


@pytest.mark.parametrize("name", ["norm_quant", "fp8_matmul", "batch_maps"])
@pytest.mark.parametrize("default", [False, True])   # from the default stream to another, and from another to the default one
def test_what_a_call_allocates_belongs_to_its_stream(kda, name, default):
    """Once dropped it is not handed out on the stream that was current, where its kernel may still be running, but
    on the call's own."""
    call = calls(kda)[name]
    other = torch.cuda.Stream()
    current, stream = (other, torch.cuda.default_stream()) if default else (torch.cuda.default_stream(), other)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(current):
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        out = call(stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a.double(), b.double()) for a, b in zip(want, out))
        blocks = {t.data_ptr(): t.untyped_storage().nbytes() for t in out if t.untyped_storage().nbytes() >= 1 << 20}
        assert blocks
        del out
        here = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in blocks.values()]
        with torch.cuda.stream(stream):
            there = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in blocks.values()]
    assert not {t.data_ptr() for t in here} & set(blocks)
    assert {t.data_ptr() for t in there} == set(blocks)


def test_results_dropped_before_their_readers_have_run(kda):
    """q and the scales pass between two calls on a busy stream and are dropped at once; what is allocated and
    written on the current stream meanwhile must not be their memory."""
    g = torch.Generator().manual_seed(43)
    x = torch.randn(4000, 2048, generator=g).to(BF16).cuda()
    w, sw = weights(640, 2048, 44)
    q, s, _ = kda.kda_norm_quant(x)
    want = kda.kda_fp8_matmul(q, s, w, sw)
    del q, s
    side = torch.cuda.Stream()
    busy = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for i in range(40):
            busy.fill_(i)
    q, s, _ = kda.kda_norm_quant(x, stream=side)
    got = kda.kda_fp8_matmul(q, s, w, sw, stream=side)
    sizes = [t.untyped_storage().nbytes() for t in (q, s)]
    del q, s
    junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    assert len(junk) == 2 and torch.equal(got, want)


# ---- offsets past 32 bits -----------------------------------------------------------------

FAR = (1 << 30) + 16   # elements from a row to the next: the third starts past 2^31


@pytest.fixture(scope="module")
def far():
    """Four buffers of 5 GB, from which rows are taken FAR elements apart."""
    bufs = [torch.zeros(5 * FAR, dtype=torch.uint8, device="cuda") for _ in range(4)]
    yield bufs
    del bufs
    torch.cuda.empty_cache()


def rows_apart(buf, t, stride):
    """The values of `t` in rows of `buf` that lie `stride` elements apart."""
    v = buf.view(t.dtype).as_strided(t.shape, (stride, 1))
    v.copy_(t)
    return v


@pytest.mark.parametrize("cols", [384, 391])
def test_norm_quant_rows_far_apart(kda, far, cols):
    x = torch.randn(2, cols, generator=torch.Generator().manual_seed(61)).to(BF16).cuda()
    w = torch.ones(cols, device="cuda")
    q, s, ro = kda.kda_norm_quant(x, w, residual=x)
    got = {"residual_out": rows_apart(far[1], torch.zeros_like(x), 2 * FAR), "q": rows_apart(far[2], torch.zeros_like(q), 4 * FAR),
           "scales": rows_apart(far[3], torch.zeros_like(s), FAR)}
    kda.kda_norm_quant(rows_apart(far[0], x, 2 * FAR), w, residual=x, **got)
    assert torch.equal(got["residual_out"], ro) and torch.equal(got["q"].float(), q.float()) and torch.equal(got["scales"], s)


@pytest.mark.parametrize("M", [5, 40, 3000])
@pytest.mark.parametrize("step", [FAR, FAR - 3])   # rows on 16-byte boundaries and off them
def test_fp8_matmul_rows_far_apart(kda, far, M, step):
    """w's rows, and with five of them a's and the output's too."""
    a, sa, w, sw = operands(M, 5, 272, 62)
    w = rows_apart(far[1], w, step)
    out = None
    if M == 5:
        a, out = rows_apart(far[0], a, step), rows_apart(far[2], torch.zeros(5, 5, dtype=BF16, device="cuda"), FAR // 2)
    assert (kda.kda_fp8_matmul_plan(a, w)[0] == 0) == (step != FAR)
    check_matmul(kda, a, sa, w, sw, out=out)
