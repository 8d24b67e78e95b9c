"""The attention side of a serving step on the GPU against oracle/attention.py:
norms with rotation and cache write (bit for bit), attention over the NVFP4
cache, operations on pages (equal), refusals, streams and far addresses."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests.helpers import require_gpu, to_np_f32

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32 = np.float32
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    import mixture_experts_layer_fwd_gb300 as m
    m.moe_sync_status()
    yield
    assert m.moe_sync_status() == 0


def moe():
    import mixture_experts_layer_fwd_gb300 as m
    return m


def dev(x, dtype=None):
    return torch.as_tensor(np.asarray(x), dtype=dtype).to(DEV)


# ------------------------------------------------------------ norms, rotation
def norm_case(T, Hq, Hkv, D, rot, interleaved, P, seed, stride=0, norm=True, kind="normal"):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, (Hq + 2 * Hkv) * D + stride)).astype(F32) * 1.5
    if kind == "edges":  # zeros, blocks of zeros, tiny and huge rows
        x[::3] *= 1e-20
        x[1::3] *= 1e15
        x[:, : D // 2] = 0
        x[0] = 0
        x[:, ::7] = -0.0
    qkv = torch.from_numpy(x).bfloat16().to(DEV)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv[:, :(Hq + 2 * Hkv) * D].split((Hq * D, Hkv * D, Hkv * D), 1))
    w = [torch.from_numpy(1 + 0.1 * rng.normal(size=D).astype(F32)).bfloat16().to(DEV) if norm else None for _ in range(2)]
    top = 5000
    ang = np.arange(top)[:, None] * 1e4 ** (-np.arange(0, rot, 2) / max(rot, 1))
    cs = np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(F32)
    pos = rng.integers(0, top, T).astype(np.int32)
    N = T // P + 3
    slots = rng.permutation(N * P)[:T].astype(np.int64)
    if T > 4:
        slots[3] = -1
    gk, gv = (rng.uniform(0.001, 0.004, Hkv).astype(F32) for _ in range(2))
    return dict(q=q, k=k, v=v, wq=w[0], wk=w[1], cs=cs, pos=pos, slots=slots, gk=gk, gv=gv, N=N)


def expected_norm(c, D, rot, interleaved, P):
    cos, sin = np.split(c["cs"][c["pos"]], 2, axis=1)
    f = lambda t: None if t is None else to_np_f32(t)  # noqa: E731
    q = oa.norm_rope(f(c["q"]), f(c["wq"]), 1e-6, cos, sin, interleaved)
    k = oa.norm_rope(f(c["k"]), f(c["wk"]), 1e-6, cos, sin, interleaved)
    v = f(c["v"])
    pool = np.zeros((c["N"], k.shape[1], oa.record_bytes(P, D)), np.uint8)
    for t, s in enumerate(c["slots"]):
        if s >= 0:
            oa.write_token(pool, s, k[t], v[t], c["gk"], c["gv"], P)
    return q, k, pool


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,interleaved,P,stride,norm,kind", [
    (1, 64, 4, 128, 128, False, 64, 0, True, "normal"),
    (2, 5, 1, 128, 64, True, 32, 8, True, "normal"),
    (67, 20, 5, 64, 32, True, 128, 0, True, "normal"),
    (33, 7, 7, 64, 64, False, 32, 16, True, "normal"),
    (40, 3, 1, 64, 16, False, 64, 0, False, "normal"),
    (301, 16, 2, 128, 128, True, 64, 0, True, "normal"),
    (19, 9, 3, 128, 0, False, 64, 0, True, "normal"),
    (50, 8, 2, 128, 128, False, 64, 0, True, "edges"),
    (50, 8, 2, 64, 48, False, 32, 0, True, "edges"),
])
def test_norm_rope_and_cache_bytes_are_the_definitions(T, Hq, Hkv, D, rot, interleaved, P, stride, norm, kind):
    c = norm_case(T, Hq, Hkv, D, rot, interleaved, P, seed=T, stride=stride, norm=norm, kind=kind)
    pool = torch.zeros(c["N"], Hkv, oa.record_bytes(P, D), dtype=torch.uint8, device=DEV)
    q, k = moe().moe_qk_norm_rope(
        c["q"], c["k"], dev(c["cs"]) if rot else None, dev(c["pos"]), wq=c["wq"], wk=c["wk"], eps=1e-6,
        interleaved=interleaved, v=c["v"], pool=pool, g_k=dev(c["gk"]), g_v=dev(c["gv"]), slots=dev(c["slots"]),
        k_out=torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV))
    eq, ek, epool = expected_norm(c, D, rot, interleaved, P)
    bits = lambda t: t.cpu().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(q), bits(torch.from_numpy(eq).bfloat16()))
    assert torch.equal(bits(k), bits(torch.from_numpy(ek).bfloat16()))
    assert np.array_equal(pool.cpu().numpy(), epool)


def test_norm_rope_without_a_cache_and_in_place():
    c = norm_case(30, 6, 2, 128, 128, False, 64, seed=5)
    q = c["q"].contiguous()
    out, k = moe().moe_qk_norm_rope(q, c["k"], dev(c["cs"]), dev(c["pos"]), wq=c["wq"], wk=c["wk"], q_out=q)
    eq, ek, _ = expected_norm(c, 128, 128, False, 64)
    assert out.data_ptr() == q.data_ptr()
    assert torch.equal(out.cpu(), torch.from_numpy(eq).bfloat16()) and torch.equal(k.cpu(), torch.from_numpy(ek).bfloat16())
    empty = moe().moe_qk_norm_rope(q[:0], c["k"][:0], dev(c["cs"]), dev(c["pos"][:0]))
    assert empty[0].shape == (0, 6, 128)


def test_norm_rope_reports_positions_and_slots_outside():
    m, c = moe(), norm_case(6, 2, 1, 64, 64, False, 32, seed=6)
    pool = torch.full((c["N"], 1, oa.record_bytes(32, 64)), 7, dtype=torch.uint8, device=DEV)
    c["slots"][:] = [c["N"] * 32, 1 << 40, -1, -5, c["N"] * 32 + 9, 1 << 62]
    kw = dict(v=c["v"], pool=pool, g_k=dev(c["gk"]), g_v=dev(c["gv"]), slots=dev(c["slots"]))
    m.moe_qk_norm_rope(c["q"], c["k"], dev(c["cs"]), dev(c["pos"]), **kw)
    assert (pool == 7).all()
    assert m.moe_sync_status() == 1 and m.moe_sync_status() == 0
    c["pos"][2], c["pos"][4] = -1, 5000  # clamped
    q, _ = m.moe_qk_norm_rope(c["q"], c["k"], dev(c["cs"]), dev(c["pos"]))
    assert m.moe_sync_status() == 1
    c["pos"][2], c["pos"][4] = 0, 4999
    assert torch.equal(q, m.moe_qk_norm_rope(c["q"], c["k"], dev(c["cs"]), dev(c["pos"]))[0])


# ------------------------------------------------------------------- attention
def attn_case(D, Hkv, G, P, qs, kvs, seed, loud=1.0, spare=2):
    """Cache bytes by the oracle's quantiser; what was never written is 0xFF (its scales are NaN)."""
    rng = np.random.default_rng(seed)
    B = len(qs)
    used = [-(-n // P) for n in kvs]
    N, M = sum(used) + spare, max(max(used), 1) + 1
    pool = np.full((N, Hkv, oa.record_bytes(P, D)), 0xFF, np.uint8)
    table = np.full((B, M), -1, np.int32)
    order, at = rng.permutation(N), 0
    gk, gv = (rng.uniform(0.001, 0.003, Hkv).astype(F32) for _ in range(2))
    from oracle import nvfp4
    for b, n in enumerate(kvs):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
        for h in range(Hkv):
            k, v = (rng.normal(size=(n, D)).astype(F32) for _ in range(2))
            k[:, rng.random(D) > 0.95] *= 3
            kq, ksf, _ = nvfp4.quantize(k, gk[h]) if n else (np.zeros((0, D // 2)), np.zeros((0, D // 16)), 0)
            vq, vsf, _ = nvfp4.quantize(v, gv[h]) if n else (np.zeros((0, D // 2)), np.zeros((0, D // 16)), 0)
            for j in range(used[b]):
                sec = oa.sections(pool[table[b, j], h], P, D)
                m = min(P, n - j * P)
                for s, src in zip(sec, (kq, ksf, vq, vsf)):
                    s[:m] = src[j * P:j * P + m]
    T = sum(qs)
    q = torch.from_numpy(rng.normal(size=(T, Hkv * G, D)).astype(F32) * loud).bfloat16()
    return dict(q=q, pool=pool, gk=gk, gv=gv, table=table, starts=np.cumsum([0] + list(qs)).astype(np.int32),
                lens=np.asarray(kvs, np.int32))


def check_attention(c, P, scale, causal=True, window=0, q_dev=None, stream=None):
    q_dev = c["q"].to(DEV) if q_dev is None else q_dev
    T, Hq, D = c["q"].shape
    lse = torch.full((T, Hq), 123.0, device=DEV)
    args = (q_dev, dev(c["pool"]), dev(c["gk"]), dev(c["gv"]), dev(c["starts"]), dev(c["lens"]), dev(c["table"]))
    out = moe().moe_kv4_attention(*args, scale=scale, causal=causal, window=window, lse=lse)
    ref, rlse, weight, all_v = oa.attention(to_np_f32(c["q"]), c["pool"], c["gk"], c["gv"], c["starts"], c["lens"], c["table"],
                                     scale, P, causal, window)
    got = to_np_f32(out).astype(np.float64)
    # bf16 output: 2^-9 of the value, doubled; P in fp16: 2^-12 of sum p |v|, and
    # the errors of scores up to ~30 summed in fp32 (2^-18) and of the exponential
    # below that: 2^-10 covers them.  Where the weights that matter meet zeros in V,
    # what is left is far below P's largest value: fp16's spacing there is 2^-24
    # for a largest value of at least 2^7, half of it lost per key: 2^-32
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * weight + 2.0 ** -32 * all_v).all()
    seen = np.isfinite(rlse)
    gl = lse.cpu().numpy()
    assert (gl[~seen] == -np.inf).all() and (got[~seen] == 0).all()
    # scores: 128 fp32 sums of terms that add up to a few hundred at most
    assert np.abs(gl[seen] - rlse[seen]).max(initial=0) <= 5e-4
    again = moe().moe_kv4_attention(*args, scale=scale, causal=causal, window=window)
    assert torch.equal(out, again)
    return out


SMALL = [1, 0, 2, 1, 3]       # few rows per sequence: 16 rows at a time
CHUNKS = [70, 1, 0, 150, 33]  # chunks: 256 rows at a time


@pytest.mark.parametrize("qs", [SMALL, CHUNKS])
@pytest.mark.parametrize("D,Hkv,G,P", [(128, 2, 4, 64), (128, 1, 16, 32), (64, 2, 5, 64), (64, 1, 1, 128), (128, 1, 3, 128),
                                       (64, 1, 16, 32)])
def test_attention_of_ragged_batches(qs, D, Hkv, G, P):
    kvs = [max(n, m) for n, m in zip(qs, (P + 1, 5, 3 * P, 2 * P, 2 * P - 1))]
    check_attention(attn_case(D, Hkv, G, P, qs, kvs, seed=D + G), P, D ** -0.5)


@pytest.mark.parametrize("qs", [SMALL, CHUNKS])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 17), (True, 128), (True, 1000)])
def test_attention_masks(qs, causal, window):
    kvs = [max(n, m) for n, m in zip(qs, (300, 5, 129, 260, 64))]
    check_attention(attn_case(64, 1, 4, 32, qs, kvs, seed=window), 32, 0.2, causal, window)


@pytest.mark.parametrize("qs", [[2, 1, 3, 1], [90, 40, 200, 9]])
def test_attention_rows_that_see_nothing(qs):
    """Fewer keys than queries: the first rows see none; no keys at all; one key."""
    kvs = [qs[0] // 2, 0, 1, qs[3]]
    out = check_attention(attn_case(128, 1, 2, 32, qs, kvs, seed=3), 32, 0.1)
    assert (out[qs[0]:qs[0] + qs[1]] == 0).all()


@pytest.mark.parametrize("qs,kvs", [([1], [1]), ([1], [64]), ([1], [65]), ([1], [3001]), ([4], [4]), ([257], [257]),
                                    ([300], [1111]), ([130], [2000])])
def test_attention_of_one_sequence(qs, kvs):
    check_attention(attn_case(128, 2, 4, 64, qs, kvs, seed=kvs[0]), 64, 128 ** -0.5)


@pytest.mark.parametrize("qs", [[1, 1, 1], [40, 70, 30]])
@pytest.mark.parametrize("scale,loud", [(0.09, 12.0), (-0.09, 1.0), (0.0, 1.0), (1e-3, 300.0)])
def test_attention_scales(qs, scale, loud):
    """Peaked rows (the maximum moves by far more than 2^8), negative and zero scales, large queries."""
    check_attention(attn_case(128, 1, 8, 64, qs, [400, 77, 513], seed=11, loud=loud), 64, scale)


@pytest.mark.parametrize("qs", [[1, 2], [60, 80]])
def test_attention_of_rising_scores(qs):
    """Keys that grow along the context: every tile brings a new maximum."""
    c = attn_case(64, 1, 2, 64, qs, [700, 640], seed=12)
    for b in range(2):
        for j in range(-(-int(c["lens"][b]) // 64)):
            oa.sections(c["pool"][c["table"][b, j], 0], 64, 64)[1][:] = 0x30 + 2 * j
    check_attention(c, 64, 0.2)


@pytest.mark.parametrize("qs", [[1, 2], [60, 80]])
@pytest.mark.parametrize("kvs", [[1500, 640], [1408, 129]])
def test_attention_of_rising_scores_on_long_contexts(qs, kvs):
    """Heads of 128: every pair of tiles moves the maximum; odd and even numbers of tiles."""
    c = attn_case(128, 1, 2, 64, qs, kvs, seed=16)
    for b in range(2):
        for j in range(-(-kvs[b] // 64)):
            oa.sections(c["pool"][c["table"][b, j], 0], 64, 128)[1][:] = 0x30 + j
    check_attention(c, 64, 0.1)


@pytest.mark.parametrize("D,P,window", [(128, 64, 0), (128, 32, 100), (128, 128, 0), (64, 64, 0)])
def test_attention_of_many_short_sequences(D, P, window):
    """Several items per block, of any number of tiles, some of them shared by two blocks, some rows empty."""
    rng = np.random.default_rng(D + P)
    qs = [int(n) for n in rng.integers(0, 3, 330)]
    kvs = [int(n) for n in rng.integers(0, 400, 330)]
    kvs[7], qs[7], kvs[200], qs[200] = 3000, 1, 0, 2
    check_attention(attn_case(D, 2, 2, P, qs, kvs, seed=17), P, D ** -0.5, window=window)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [2, 3, 4])
def test_attention_of_few_tokens_of_many_heads(D, n):
    """32, 48 and 64 rows per sequence and kv head, on either side of the kernels' border."""
    check_attention(attn_case(D, 1, 16, 64, [n] * 3, [n, 70, 391], seed=18), 64, D ** -0.5)


@pytest.mark.parametrize("qs", [[1, 2, 1], [50, 1, 99]])
def test_attention_queries_are_slices_on_another_stream(qs):
    c = attn_case(128, 1, 4, 64, qs, [200, 130, 99], seed=13)
    want = check_attention(c, 64, 0.1)
    T, Hq, D = c["q"].shape
    wide = torch.zeros(T, (Hq + 2) * D + 8, dtype=torch.bfloat16, device=DEV)
    q = wide[:, :Hq * D].unflatten(1, (Hq, D))
    q.copy_(c["q"])
    check_attention(c, 64, 0.1, q_dev=q)
    args = [q, dev(c["pool"]), dev(c["gk"]), dev(c["gv"]), dev(c["starts"]), dev(c["lens"]), dev(c["table"])]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = moe().moe_kv4_attention(*args, scale=0.1, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("qs", [[1, 1], [100, 30]])
def test_attention_reads_far_pages(qs):
    """Pages past 4 GiB of one layer's pool."""
    c = attn_case(128, 1, 2, 64, qs, [150, 100], seed=14)
    rec = oa.record_bytes(64, 128)
    N = (5 << 30) // rec
    pool = torch.empty(N, 1, rec, dtype=torch.uint8, device=DEV)
    n = c["pool"].shape[0]
    pool[N - n:] = dev(c["pool"])
    want = check_attention(c, 64, 0.1)
    far = np.where(c["table"] >= 0, c["table"] + N - n, -1).astype(np.int32)
    out = moe().moe_kv4_attention(c["q"].to(DEV), pool, dev(c["gk"]), dev(c["gv"]), dev(c["starts"]), dev(c["lens"]),
                                  dev(far), scale=0.1)
    assert torch.equal(out, want)


@pytest.mark.parametrize("qs", [[1, 1, 1], [100, 30, 20]])
def test_attention_reports_pages_outside_and_bounds_its_inputs(qs):
    m, c = moe(), attn_case(64, 1, 2, 32, qs, [150, 100, 60], seed=15)
    want = check_attention(c, 32, 0.1)
    bad = c["table"].copy()
    bad[1, 0], bad[1, 2] = -7, 1 << 30
    a = [c["q"].to(DEV), dev(c["pool"]), dev(c["gk"]), dev(c["gv"]), dev(c["starts"]), dev(c["lens"]), dev(bad)]
    out = m.moe_kv4_attention(*a, scale=0.1)
    assert m.moe_sync_status() == 1
    t0, t1 = c["starts"][1], c["starts"][2]
    assert torch.equal(out[:t0], want[:t0]) and torch.equal(out[t1:], want[t1:])  # the others are untouched
    # lengths past the table and offsets that fall or leave q stay inside the buffers
    a[6] = dev(c["table"])
    a[5] = dev(np.array([1 << 30, -4, 60], np.int32))
    a[4] = dev(np.array([-9, 1 << 30, 3, 1 << 20], np.int32))
    m.moe_kv4_attention(*a, scale=0.1)
    m.moe_sync_status()  # a table entry of -1 is met and reported


def test_attention_of_nothing():
    c = attn_case(64, 1, 2, 32, [1], [5], seed=1)
    a = [dev(c["pool"]), dev(c["gk"]), dev(c["gv"])]
    out = moe().moe_kv4_attention(c["q"][:0].to(DEV), *a, dev(np.zeros(2, np.int32)), dev(c["lens"]), dev(c["table"]))
    assert out.shape == (0, 2, 64)


# ----------------------------------------------------------------------- pages
def fill(rng, S, M, N, P, layers, Hkv=1, D=64):
    """A pool in use: rows of random lengths, some forked from others, some ended."""
    s = oa.Pages([[-1] * M for _ in range(S)], [0] * S, [0] * N, P)
    s.extend([int(n) for n in rng.integers(0, max(1, (M - 1) * P), S) * (rng.random(S) < 0.6)])
    empty = [r for r in range(S) if s.lens[r] == 0]
    full = [r for r in range(S) if s.lens[r] > 0]
    if full:
        s.fork([int(rng.choice(full)) for _ in empty[::2]], empty[::2])
        s.free([int(r) for r in rng.choice(full, max(1, len(full) // 3))])
    pool = rng.integers(0, 256, (layers, N, Hkv, oa.record_bytes(P, D)), dtype=np.uint8)
    return s, pool


def state(s):
    return dev(s.table, I32), dev(s.lens, I32), dev(s.refs, I32)


def same(o, s):
    assert o["table"].cpu().tolist() == s.table
    assert o["refs"].cpu().tolist() == s.refs
    if "lens" in o:
        assert o["lens"].cpu().tolist() == s.lens


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("S,M,N,P", [(1, 1, 1, 32), (7, 5, 40, 32), (300, 9, 1500, 64), (40, 40, 20001, 128)])
def test_page_operations_against_lists(S, M, N, P, inplace):
    m = moe()
    for seed in range(3):
        rng = np.random.default_rng(seed * 10 + S)
        s, pool = fill(rng, S, M, N, P, layers=2)
        d_pool = dev(pool)
        # extend
        table, lens, refs = state(s)
        counts = [int(n) for n in rng.integers(0, P, S) * (rng.random(S) < 0.7)]
        slots, pos, failed = s.extend(counts)
        keep = table.clone(), lens.clone(), refs.clone()
        o = m.moe_kv_extend(dev(np.cumsum([0] + counts), I32), sum(counts), table, lens, refs, P, inplace=inplace)
        same(o, s)
        assert o["slots"].cpu().tolist() == slots and o["pos"].cpu().tolist() == pos
        assert (m.moe_sync_status() != 0) == bool(failed)
        if not inplace:
            assert all(torch.equal(a, b) for a, b in zip(keep, (table, lens, refs)))
        # fork
        empty, full = [r for r in range(S) if not s.lens[r]], [r for r in range(S) if s.lens[r]]
        if empty and full:
            dst = empty[:max(1, len(empty) // 2)]
            src = [int(rng.choice(full)) for _ in dst]
            table, lens, refs = state(s)
            short = len(s.free_pages())
            need = sum(s.lens[r] % P > 0 for r in src)
            for a, b in s.fork(src, dst):
                pool[:, b] = pool[:, a]
            o = m.moe_kv_fork(dev(src, I32), dev(dst, I32), table, lens, refs, d_pool, page_size=P, inplace=inplace)
            same(o, s)
            assert np.array_equal(d_pool.cpu().numpy(), pool)
            assert m.moe_sync_status() == (6 if need > short else 0)
        # free
        table, lens, refs = state(s)
        rows = [int(r) for r in rng.integers(0, S, max(1, S // 3))]  # some twice
        s.free(rows)
        same(m.moe_kv_free(dev(rows, I32), table, lens, refs, page_size=P, inplace=inplace), s)
        # compact
        table, lens, refs = state(s)
        remap, moves = s.compact()
        for a, b in moves:
            pool[:, b] = pool[:, a]
        o = m.moe_kv_compact(table, refs, d_pool, inplace=inplace)
        same(o, s)
        assert o["remap"].cpu().tolist() == remap
        assert np.array_equal(d_pool.cpu().numpy(), pool)
        assert m.moe_sync_status() == 0


def test_extend_out_of_pages_and_out_of_room():
    m, P = moe(), 32
    s = oa.Pages([[-1] * 2 for _ in range(4)], [0] * 4, [0] * 4, P)
    for counts, want in (([40, 0, 33, 0], 0), ([0, 5, 0, 64], 6), ([20, 0, 40, 0], 1), ([24, 0, 0, 0], 1)):
        table, lens, refs = state(s)
        slots, pos, failed = s.extend(counts)
        o = m.moe_kv_extend(dev(np.cumsum([0] + counts), I32), sum(counts), table, lens, refs, P)
        same(o, s)
        assert o["slots"].cpu().tolist() == slots
        assert m.moe_sync_status() == want


def test_fork_leaves_out_pairs_that_are_not_allowed():
    m, P = moe(), 32
    s = oa.Pages([[-1] * 3 for _ in range(6)], [0] * 6, [0] * 20, P)
    s.extend([50, 64, 0, 0, 0, 0])
    table, lens, refs = state(s)
    s.fork([0, 1], [2, 3])  # the others: dst in use, dst twice, rows that are not there
    o = m.moe_kv_fork(dev([0, 0, 1, 0, -1, 0], I32), dev([2, 1, 3, 2, 4, 6], I32), table, lens, refs, page_size=P)
    same(o, s)
    assert m.moe_sync_status() == 1


@pytest.mark.parametrize("layers,n,pages", [(1, 1, 2), (3, 7, 40), (2, 60, 200)])
def test_copy_pages(layers, n, pages):
    m, rng = moe(), np.random.default_rng(n)
    pool = rng.integers(0, 256, (layers, pages, 2, oa.record_bytes(64, 128)), dtype=np.uint8)
    order = rng.permutation(pages)
    src, dst = order[:n], order[n:2 * n]
    d = dev(pool)
    m.moe_kv_copy_pages(d, dev(src, I32), dev(dst, I32))
    pool[:, dst] = pool[:, src]
    assert np.array_equal(d.cpu().numpy(), pool)
    m.moe_kv_copy_pages(d, dev([0, -1, pages], I32), dev([pages, 1, 0], I32))
    assert m.moe_sync_status() == 1 and np.array_equal(d.cpu().numpy(), pool)


def test_copy_of_far_pages():
    rec = oa.record_bytes(64, 128)
    N = (5 << 30) // rec
    pool = torch.empty(1, N, 1, rec, dtype=torch.uint8, device=DEV)
    pool[0, N - 1] = torch.arange(rec, device=DEV) % 251
    moe().moe_kv_copy_pages(pool, dev([N - 1], I32), dev([N - 2], I32))
    assert torch.equal(pool[0, N - 2], pool[0, N - 1])


# ---------------------------------------------------------------------- refusals
def test_refusals_of_the_binding():
    m = moe()
    bf = dict(dtype=torch.bfloat16, device=DEV)
    q, k = torch.zeros(4, 8, 64, **bf), torch.zeros(4, 2, 64, **bf)
    with pytest.raises(TypeError, match="q"):
        m.moe_qk_norm_rope(q.float(), k)
    with pytest.raises(ValueError, match="contiguous within a token"):
        m.moe_qk_norm_rope(q.transpose(0, 1), torch.zeros(8, 2, 64, **bf))
    with pytest.raises(ValueError, match="head size"):
        m.moe_qk_norm_rope(q, torch.zeros(4, 2, 128, **bf))
    with pytest.raises(ValueError, match="pos: required"):
        m.moe_qk_norm_rope(q, k, torch.zeros(9, 64, device=DEV))
    pool = torch.zeros(3, 2, oa.record_bytes(64, 64), dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError, match="v: required"):
        m.moe_qk_norm_rope(q, k, pool=pool)
    with pytest.raises(m._lib.MoEError):  # head size without a kernel
        m.moe_qk_norm_rope(torch.zeros(4, 8, 96, **bf), torch.zeros(4, 2, 96, **bf))
    with pytest.raises(m._lib.MoEError):  # rotation not a multiple of 16
        m.moe_qk_norm_rope(q, k, torch.zeros(9, 24, device=DEV), torch.zeros(4, dtype=I32, device=DEV))
    g = torch.ones(2, device=DEV)
    i = lambda *s: torch.zeros(*s, dtype=I32, device=DEV)  # noqa: E731
    with pytest.raises(ValueError, match="pool"):
        m.moe_kv4_attention(q, pool[:, :1].contiguous(), g, g, i(2), i(1), i(1, 1))
    with pytest.raises(ValueError, match="q_offsets"):
        m.moe_kv4_attention(q, pool, g, g, i(3), i(1), i(1, 1))
    with pytest.raises(m._lib.MoEError):  # a window without causality
        m.moe_kv4_attention(q, pool, g, g, i(2), i(1), i(1, 1), causal=False, window=4)
    with pytest.raises(m._lib.MoEError):  # too little workspace
        m.moe_kv4_attention(q, pool, g, g, i(2), i(1), i(1, 1), ws=torch.zeros(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="lens"):
        m.moe_kv_free(i(1), i(4, 2), i(3), i(8))
    with pytest.raises(m._lib.MoEError):  # page size without a kernel
        m.moe_kv_free(i(1), i(4, 2), i(4), i(8), page_size=48)
