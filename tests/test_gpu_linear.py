"""Products of a few tokens with an NVFP4 matrix on the GPU against the formula
in 64 bits: sizes around the kernel's tiles, strides, ranges, refusals, streams
and graphs."""
import numpy as np
import pytest
import torch

from oracle import nvfp4
from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def moe():
    import mixture_experts_layer_fwd_gb300 as m
    return m


def case(T, N, K, seed=0, kind="normal"):
    rng = np.random.default_rng(seed + 1000 * T + N + K)
    x = rng.normal(size=(T, K)).astype(np.float32)
    if kind == "edges":  # tokens of very different sizes, values of very different sizes in one token
        x *= (10.0 ** rng.integers(-30, 30, size=(T, 1))).astype(np.float32)
        x *= (2.0 ** -rng.integers(0, 45, size=(T, K))).astype(np.float32)
        x[0, ::3] = 0
    codes = rng.integers(0, 256, size=(N, K // 2)).astype(np.uint8)
    sf = rng.integers(0, 0x7F, size=(N, K // 16)).astype(np.uint8)  # zero, subnormal, up to 448
    if kind == "edges":
        sf[::2] |= 0x80
    g = np.float32(0.37 if kind == "normal" else 3e-4)
    return torch.from_numpy(x).bfloat16(), codes, sf, g


def expected(x, codes, sf, g, add=None):
    """The formula in 64 bits, and how far fp32 sums may be off: every one of K / 16
    instructions adds 16 products and the sum so far with 2^-22 of their magnitude
    (truncated alignment of 17 terms), joining 16 parts as much again; values below
    2^-29 of a token's largest are off by 2^-40 of it."""
    w = nvfp4.dequantize(codes, sf, g)
    xd = x.double().numpy()
    y, size = xd @ w.T, np.abs(xd) @ np.abs(w).T
    K = xd.shape[1]
    off = (K / 16 + 16) * 2.0 ** -22 * size + 2.0 ** -40 * np.abs(xd).max(1, keepdims=True) * np.abs(w).sum(1)
    if add is not None:
        a = add.double().numpy()
        y, off = y + a, off + 2.0 ** -24 * np.abs(a)
    return y, off + 2.0 ** -23 * np.abs(y) + 1e-37


def check(out, y, off):
    got = out.double().cpu().numpy()
    if out.dtype == torch.bfloat16:
        off = off + 2.0 ** -8 * (np.abs(y) + off)
    bad = np.abs(got - y) > off
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], got[bad][:4], y[bad][:4], off[bad][:4])


def put(x, codes, sf, g):
    return x.to(DEV), torch.from_numpy(codes).to(DEV), torch.from_numpy(sf).to(DEV), torch.tensor([g], device=DEV)


SIZES = [(1, 1, 32), (1, 16, 64), (3, 17, 96), (2, 15, 288), (5, 100, 256), (8, 1024, 4096), (1, 2433, 1056), (9, 333, 544),
         (16, 600, 8192), (17, 50, 2080), (24, 260, 4096), (32, 77, 16384), (31, 5000, 1024), (2, 40000, 512), (25, 16, 32),
         (7, 2432, 7168), (32, 4865, 320), (8, 70, 16640), (9, 31, 256), (3, 129, 65536), (32, 300, 32768), (20, 33, 30976)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("f32", [False, True])
def test_linear_is_the_formula(T, N, K, f32):
    a = case(T, N, K)
    out = moe().moe_linear_nvfp4(*put(*a), out_dtype=torch.float32 if f32 else torch.bfloat16)
    assert out.shape == (T, N)
    check(out, *expected(*a))


@pytest.mark.parametrize("T,N,K", [(32, 155000, 1280), (17, 60001, 2304), (24, 79000, 4096), (8, 90000, 1024), (1, 200000, 768)])
def test_linear_of_many_rows(T, N, K):
    """More rows than a round of the blocks, tokens that come a chunk at a time: a sample
    of them against the formula."""
    x, codes, sf, g = case(T, N, K)
    d = put(x, codes, sf, g)
    out = moe().moe_linear_nvfp4(*d, out_dtype=torch.float32)
    rows = np.unique(np.concatenate((np.arange(40), np.arange(N - 70, N), np.random.default_rng(1).integers(0, N, 3000))))
    check(out[:, rows], *expected(x, codes[rows], sf[rows], g))
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("T,N,K", [(1, 100, 512), (6, 33, 1056), (12, 64, 256), (32, 40, 4160)])
def test_linear_keeps_the_range_of_its_types(T, N, K):
    a = case(T, N, K, kind="edges")
    out = moe().moe_linear_nvfp4(*put(*a), out_dtype=torch.float32)
    check(out, *expected(*a))


@pytest.mark.parametrize("T,N,K", [(1, 100, 512), (4, 70, 2080), (16, 40, 4096), (16, 33, 288), (17, 40, 4096), (32, 33, 288)])
@pytest.mark.parametrize("top", [-90, -4, 0, 6, 15, 90])
@pytest.mark.parametrize("deep", [False, True])
def test_small_values_beside_a_large_one_that_meets_no_weight(T, N, K, top, deep):
    """However many tokens: exact down to 2^-29 of a token's largest value, off by 2^-40 of it at most below."""
    rng = np.random.default_rng(T + K + top)
    x = rng.uniform(1, 2, size=(T, K)) * 2.0 ** (top - rng.integers(*((30, 40) if deep else (20, 30)), size=(T, K)))
    x = (x * rng.choice([-1, 1], size=x.shape)).astype(np.float32)
    x[:, :16] = 0
    x[:, 5] = 2.0 ** top
    _, codes, sf, g = case(T, N, K)
    sf[:, 0] = 0
    x = torch.from_numpy(x).bfloat16()
    w, xd = nvfp4.dequantize(codes, sf, g), x.double().numpy()
    y, size = xd @ w.T, np.abs(xd) @ np.abs(w).T  # the large value is in neither
    off = (K / 16 + 16) * 2.0 ** -22 * size + 2.0 ** -23 * np.abs(y)  # as in expected()
    if deep:
        off = off + 2.0 ** (top - 40) * np.abs(w).sum(1)
    check(moe().moe_linear_nvfp4(*put(x, codes, sf, g), out_dtype=torch.float32), y, off)


@pytest.mark.parametrize("T,N,K", [(1, 64, 128), (4, 130, 160), (20, 48, 1024)])
@pytest.mark.parametrize("f32", [False, True])
def test_linear_adds_and_takes_strided_rows(T, N, K, f32):
    x, codes, sf, g = case(T, N, K)
    wide = torch.zeros(T, K + 24, dtype=torch.bfloat16, device=DEV)
    wide[:, 8:8 + K] = x.to(DEV)
    add = torch.randn(T, 3 * N + 1, generator=torch.Generator().manual_seed(1)).bfloat16()[:, N:2 * N]
    _, c, s, gg = put(x, codes, sf, g)
    out = moe().moe_linear_nvfp4(wide[:, 8:8 + K], c, s, gg, add=add.to(DEV), out_dtype=torch.float32 if f32 else torch.bfloat16)
    check(out, *expected(x, codes, sf, g, add))


def test_linear_may_write_over_what_it_adds():
    x, codes, sf, g = case(5, 300, 512)
    add = torch.randn(5, 300, generator=torch.Generator().manual_seed(2)).bfloat16()
    at = add.to(DEV)
    out = moe().moe_linear_nvfp4(*put(x, codes, sf, g), add=at, out=at)
    assert out.data_ptr() == at.data_ptr()
    check(out, *expected(x, codes, sf, g, add))


def test_linear_of_matrices_off_the_32_byte_boundary():
    x, codes, sf, g = case(3, 40, 256)
    d = put(x, codes, sf, g)
    room = torch.empty(40 * 128 + 16, dtype=torch.uint8, device=DEV)
    c = room[16:].view(40, 128)
    c.copy_(d[1])
    check(moe().moe_linear_nvfp4(d[0], c, d[2], d[3], out_dtype=torch.float32), *expected(x, codes, sf, g))


def test_a_token_that_is_not_a_number_touches_its_own_outputs_alone():
    x, codes, sf, g = case(4, 50, 512)
    good = moe().moe_linear_nvfp4(*put(x, codes, sf, g), out_dtype=torch.float32)
    x[1, 77], x[3, 0] = float("nan"), float("inf")
    out = moe().moe_linear_nvfp4(*put(x, codes, sf, g), out_dtype=torch.float32)
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    assert out[1].isnan().all() and not out[3].isfinite().all()


def test_linear_gives_the_same_bits_each_time_on_any_stream_and_in_a_graph():
    m, a = moe(), put(*case(6, 1000, 2048))
    want = m.moe_linear_nvfp4(*a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = m.moe_linear_nvfp4(*a, stream=s)
    with torch.cuda.stream(s):
        got2 = m.moe_linear_nvfp4(*a)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got2, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_linear_nvfp4(*a, out=out)
    a[0].copy_(a[0].flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want.flip(0))


def test_linear_refuses():
    m = moe()
    x, c, s, g = put(*case(4, 32, 64))
    assert m.moe_linear_nvfp4(x[:0], c, s, g).shape == (0, 32)
    assert m.moe_linear_nvfp4(x, c[:0], s[:0], g).shape == (4, 0)
    for bad, error in (((x.float(), c, s, g), TypeError), ((x[:, :48], c, s, g), ValueError), ((x.T, c, s, g), ValueError),
                       ((x, c[:, :16], s, g), ValueError), ((x, c, s[:3], g), ValueError), ((x, c, s, g.double()), TypeError),
                       ((x.cpu(), c, s, g), ValueError), ((x, c.int(), s, g), TypeError), ((x, c, None, g), ValueError)):
        with pytest.raises(error):
            m.moe_linear_nvfp4(*bad)
    with pytest.raises(TypeError):
        m.moe_linear_nvfp4(x, c, s, g, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        m.moe_linear_nvfp4(x, c, s, g, add=torch.zeros(4, 31, device=DEV).bfloat16())
    with pytest.raises(TypeError):
        m.moe_linear_nvfp4(x, c, s, g, out=torch.empty(4, 32, device=DEV))
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        m.moe_linear_nvfp4(torch.zeros(33, 64, device=DEV).bfloat16(), c, s, g)
    with pytest.raises(RuntimeError, match="INVALID"):  # a token off the 16-byte boundary
        m.moe_linear_nvfp4(torch.zeros(4, 68, device=DEV).bfloat16()[:, 1:65], c, s, g)


@pytest.mark.parametrize("limit_ns", [1, 3000])
@pytest.mark.parametrize("T,N,K", [(3, 40000, 1024), (24, 79000, 2560), (16, 600, 8192), (20, 4096, 16384)])
def test_linear_that_gives_up_stays_inside_its_buffers(T, N, K, limit_ns):
    """The next call is right again."""
    m = moe()
    x, codes, sf, g = case(T, 8, K)
    gen = torch.Generator(DEV).manual_seed(N)
    a = (x.to(DEV), torch.randint(0, 256, (N, K // 2), generator=gen, device=DEV, dtype=torch.uint8),
         torch.randint(0, 0x70, (N, K // 16), generator=gen, device=DEV, dtype=torch.uint8), torch.tensor([0.5], device=DEV))
    want, guard = m.moe_linear_nvfp4(*a, out_dtype=torch.float32), 1 << 16
    assert torch.isfinite(want).all()
    outs = torch.full((T * N + 2 * guard,), 3.0, device=DEV)
    try:
        m.moe_set_wait_timeout_ns(limit_ns)
        m.moe_linear_nvfp4(*a, out=outs[guard:-guard].view(T, N), out_dtype=torch.float32)
    finally:
        m.moe_set_wait_timeout_ns(0)
    assert m.moe_sync_status() in (0, 5)
    assert (outs[:guard] == 3.0).all() and (outs[-guard:] == 3.0).all()
    assert torch.equal(m.moe_linear_nvfp4(*a, out_dtype=torch.float32), want) and m.moe_sync_status() == 0
