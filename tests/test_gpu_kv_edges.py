"""Edges of the cache calls on the GPU: waits that run out, odd offsets, no rows,
windows without an end, NaN, steps that were overtaken, graphs and threads."""
import threading

import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests.helpers import require_gpu, to_np_f32
from tests.test_gpu_kv4 import DEV, F32, I32, attn_case, dev, same, state
from tests.test_gpu_kv_cache import LAYERS, bytes_of, cache, inputs, run

pytestmark = pytest.mark.gpu


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


def attn_args(c):
    return (c["q"].to(DEV), dev(c["pool"]), dev(c["gk"]), dev(c["gv"]), dev(c["starts"]), dev(c["lens"]), dev(c["table"]))


# heads, new tokens of each sequence: the 16-row kernel, the decode kernel that
# makes its own schedule, the one with a schedule in front, the 256-row kernel
KERNELS = [(64, [1, 2]), (128, [1, 2]), (128, [1] * 40), (64, [300, 90]), (128, [300, 90])]


# ------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("lazy", [False, True])
@pytest.mark.parametrize("limit_us", [1000, 20000])
def test_attention_waits_give_up_near_their_limit(lazy, limit_us):
    """They count tests of about 4 us (5 % more where they sleep in between): within a factor of two of the limit."""
    m = moe()
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    m.moe_selftest_attention_wait_timeout(1000, lazy)  # the first launch loads the kernel
    assert m.moe_sync_status() == 5
    t[0].record()
    m.moe_selftest_attention_wait_timeout(1000 * limit_us, lazy)
    t[1].record()
    assert m.moe_sync_status() == 5 and m.moe_sync_status() == 0
    assert limit_us / 2 <= 1000 * t[0].elapsed_time(t[1]) <= 2 * limit_us


@pytest.mark.parametrize("limit_us", [0, 20, 60])
@pytest.mark.parametrize("D,qs,kv", [
    (64, [1] * 40, 8192),     # the 16-row kernel
    (128, [1] * 15, 16384),   # the decode kernel that makes its own schedule
    (128, [1] * 40, 8192),    # the one with a schedule in front
    (64, [300, 90], 16384),   # the 256-row kernel
    (128, [300, 90], 16384),
])
def test_attention_that_gives_up_stays_inside_its_buffers(D, qs, kv, limit_us):
    """Whatever the workspace held before; the next call is right again.  Every
    block has some 10 us of work and more copies than its ring takes: with no
    time to wait it gives up, with more it may get through."""
    m, Hkv, G, P = moe(), 2, 4, 64
    T, B, Hq = sum(qs), len(qs), Hkv * G
    gen = torch.Generator(DEV).manual_seed(21)
    pool = torch.randint(0, 256, (64, Hkv, oa.record_bytes(P, D)), generator=gen, device=DEV, dtype=torch.uint8)
    for first in (P * D // 2, P * D // 16 * 9 + P * D // 2):
        pool[:, :, first:first + P * D // 16] = 0x38
    g = torch.full((Hkv,), 0.01, device=DEV)
    q = torch.randn(T, Hq, D, generator=gen, device=DEV).bfloat16()
    args = (q, pool, g, g, dev(np.cumsum([0] + qs), I32), dev([kv - 5 * (i % 3) for i in range(B)], I32),
            torch.randint(0, 64, (B, kv // P), generator=gen, device=DEV, dtype=I32))
    want = m.moe_kv4_attention(*args)
    assert torch.isfinite(want).all()
    n, guard = want.numel(), 1 << 16
    outs = torch.full((n + 2 * guard,), 3.0, dtype=torch.bfloat16, device=DEV)
    lses = torch.full((T * Hq + 2 * guard,), 3.0, device=DEV)
    size = m._lib.load().moe_kv4_attention_workspace_size(T, B, Hq, Hkv, D)
    wss = torch.full((size + 2 * guard,), 0x7F, dtype=torch.uint8, device=DEV)
    out, lse, ws = (t[guard:t.numel() - guard] for t in (outs, lses, wss))
    try:
        m.moe_set_wait_timeout_ns(max(1, 1000 * limit_us))
        m.moe_kv4_attention(*args, out=out.view(want.shape), lse=lse.view(T, Hq), ws=ws)
    finally:
        m.moe_set_wait_timeout_ns(0)
    status = m.moe_sync_status()
    assert status == 5 or (status == 0 and limit_us > 0)
    for t, v in ((outs, 3.0), (lses, 3.0), (wss, 0x7F)):
        assert (t[:guard] == v).all() and (t[t.numel() - guard:] == v).all()
    assert torch.equal(m.moe_kv4_attention(*args, ws=ws), want)
    assert m.moe_sync_status() == 0


# ------------------------------------------------------------------- the class
@pytest.mark.parametrize("what", ["fork", "free", "compact"])
def test_a_step_is_over_once_rows_or_pages_have_moved(what):
    """Its slots may be another row's by then: nothing is written until the next extend."""
    q, k, v, cs = inputs(40)
    c = cache()
    run(c, 0, 5, q, k, v, cs, [40])
    run(c, 1, 5, q, k, v, cs, [33])
    c.extend([1, 0, 0, 0, 0])
    {"fork": lambda: c.fork([0], [2]), "free": lambda: c.free([1]), "compact": c.compact}[what]()
    keep = c.pool.clone()
    with pytest.raises(ValueError, match="extend"):
        c.attend(0, q[:1], k[:1], v[:1], cs)
    assert torch.equal(c.pool, keep)
    c.extend([1, 0, 0, 0, 0])
    for layer in range(LAYERS):
        c.attend(layer, q[:1], k[:1], v[:1], cs)
    assert moe().moe_sync_status() == 0


@pytest.mark.parametrize("counts", [[3, -1, 0, 0, 0], [1, 2], [0] * 6])
def test_counts_are_one_per_row_and_not_negative(counts):
    c = cache()
    with pytest.raises(ValueError, match="counts"):
        c.extend(counts)
    assert c.lens.tolist() == [0] * 5 and int(c.refs.sum()) == 0


def test_a_row_without_room_gets_no_answer():
    """Its queries see nothing, as long as it has no place for their keys; the other rows' answers stay."""
    m = moe()
    q, k, v, cs = inputs(100)
    a, b = cache(pages=3), cache(pages=40)
    for c in (a, b):
        run(c, 0, 5, q, k, v, cs, [30])
        run(c, 1, 5, q, k, v, cs, [31])
    counts = [1, 40, 0, 2, 0]  # one page is left: row 1 needs two, row 3 one that is handed out after them
    ys = []
    for c in (a, b):
        c.extend(counts)
        ys.append(c.attend(0, q[:43], k[:43], v[:43], cs))
    assert m.moe_sync_status() == 6
    assert a.lens.tolist() == [31, 31, 0, 0, 0] and b.lens.tolist() == [31, 71, 0, 2, 0]
    assert torch.equal(ys[0][:1], ys[1][:1]) and (ys[0][1:] == 0).all() and (ys[1][1:] != 0).any()
    a.free([1])
    a.extend([1, 0, 0, 2, 0])
    b.extend([1, 0, 0, 0, 0])
    y = a.attend(0, q[:3], k[:3], v[:3], cs)
    assert torch.equal(y[:1], b.attend(0, q[:1], k[:1], v[:1], cs)) and (y[1:] != 0).any()
    assert m.moe_sync_status() == 0
    a.extend([0] * 5)  # a step without tokens
    assert a.attend(0, q[:0], k[:0], v[:0], cs).shape[0] == 0


# ---------------------------------------------------------------------- extend
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("rows,T,offsets", [
    (3, 90, [7, 20, 20, 60]),           # tokens in front of the rows and behind them
    (3, 90, [90, 90, 90, 90]),
    (4, 90, [5, 40, 10, 70, 60]),       # offsets that fall
    (4, 90, [-9, 30, 1 << 30, 3, -1]),  # and leave the tokens
    (2500, 6000, None),                 # more rows than a block has threads
])
def test_extend_reads_its_offsets_as_attention_does(rows, T, offsets, inplace):
    """Inside the tokens and never falling; a token that no row has goes nowhere."""
    m, P = moe(), 32
    rng = np.random.default_rng(rows)
    if offsets is None:
        offsets = np.sort(rng.integers(11, T - 7, rows + 1))
        offsets[rng.integers(0, rows, 200)] -= 300
    used = np.maximum.accumulate(np.clip(offsets, 0, T))
    s = oa.Pages([[-1] * 9 for _ in range(rows)], [0] * rows, [0] * (rows + 400), P)
    s.extend([3 * (r % 5) for r in range(rows)])
    table, lens, refs = state(s)
    slots, pos, failed = s.extend([int(n) for n in np.diff(used)])
    assert not failed
    before, after = int(used[0]), T - int(used[-1])
    junk = dict(slots=torch.full((T,), 5, dtype=torch.int64, device=DEV), pos=torch.full((T,), 7, dtype=I32, device=DEV))
    o = m.moe_kv_extend(dev(offsets, I32), T, table, lens, refs, P, inplace=inplace, out=junk)
    same(o, s)
    assert o["slots"].cpu().tolist() == [-1] * before + slots + [-1] * after
    assert o["pos"].cpu().tolist() == [0] * before + pos + [0] * after


# --------------------------------------------------------------------- no rows
def test_page_operations_of_no_rows():
    m = moe()
    i = lambda *s: torch.zeros(*s, dtype=I32, device=DEV)  # noqa: E731
    refs = dev([3, 0, 1, 0, 2, 0, 0, 0], I32)
    junk = lambda: dict(refs=torch.full((8,), 77, dtype=I32, device=DEV))  # noqa: E731
    slots, pos = torch.full((5,), 9, dtype=torch.int64, device=DEV), torch.full((5,), 9, dtype=I32, device=DEV)
    o = m.moe_kv_extend(dev([2], I32), 5, i(0, 4), i(0), refs, 32, out=dict(junk(), slots=slots, pos=pos))
    assert torch.equal(o["refs"], refs) and o["slots"].tolist() == [-1] * 5 and o["pos"].tolist() == [0] * 5
    assert m.moe_kv_extend(dev([0], I32), 0, i(0, 4), i(0), refs, 32, out=junk())["refs"].equal(refs)
    assert m.moe_kv_fork(i(0), i(0), i(0, 4), i(0), refs, out=junk())["refs"].equal(refs)
    assert m.moe_kv_free(i(0), i(0, 4), i(0), refs, out=junk())["refs"].equal(refs)
    with pytest.raises(ValueError, match="no rows"):
        m.moe_kv_fork(i(1), i(1), i(0, 4), i(0), refs)
    with pytest.raises(ValueError, match="no rows"):
        m.moe_kv_free(i(1), i(0, 4), i(0), refs)
    o = m.moe_kv_compact(i(0, 4), refs, out=junk())
    assert o["refs"].tolist() == [3, 2, 1, 0, 0, 0, 0, 0] and o["remap"].tolist() == [0, -1, 2, -1, 1, -1, -1, -1]
    assert m.moe_sync_status() == 0


# --------------------------------------------------------------------- windows
@pytest.mark.parametrize("D,qs", [(64, [3, 1]), (128, [3, 1]), (64, [400, 1]), (128, [400, 1])])
def test_a_window_that_never_ends_is_none(D, qs):
    """Also where a sequence has more queries than keys and these fill several tiles."""
    m = moe()
    c = attn_case(D, 1, 16 if qs[0] < 100 else 1, 32, qs, [max(2, qs[0] - 90), 300], seed=22)
    args = attn_args(c)
    want = m.moe_kv4_attention(*args, scale=0.1)
    for window in (2 ** 31 - 1, 2 ** 31 - 9, 2 ** 31, 2 ** 32 + 5, 1 << 30):
        assert torch.equal(m.moe_kv4_attention(*args, scale=0.1, window=window), want)


# -------------------------------------------------------------------------- NaN
def check_poisoned(c, clean, out, lse, poisoned, P, scale):
    """Rows (token, head) in `poisoned` are NaN throughout, the others within the bound of tests/test_gpu_kv4.py."""
    ref, rlse, weight, all_v = oa.attention(to_np_f32(clean["q"]), clean["pool"], c["gk"], c["gv"], c["starts"], c["lens"],
                                            c["table"], scale, P, True, 0)
    got, gl = to_np_f32(out).astype(np.float64), lse.cpu().numpy()
    assert np.isnan(got[poisoned]).all() and np.isnan(gl[poisoned]).all()
    bad = np.abs(got - ref) > 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * weight + 2.0 ** -32 * all_v
    assert not bad[~poisoned].any() and not np.isnan(got[~poisoned]).any()
    assert np.abs(gl[~poisoned] - rlse[~poisoned]).max(initial=0) <= 5e-4


@pytest.mark.parametrize("kv", [100, 3000])  # one block's, and many blocks'
@pytest.mark.parametrize("D,qs", KERNELS)
def test_a_query_that_is_not_a_number_answers_with_none(D, qs, kv):
    clean = attn_case(D, 2, 4, 64, qs, [max(kv, n) for n in qs], seed=23)
    c = dict(clean, q=clean["q"].clone())
    T, Hq, _ = c["q"].shape
    poisoned = np.zeros((T, Hq), bool)
    poisoned[0, 1] = poisoned[T - 1, 6] = True
    c["q"][0, 1, 3] = c["q"][T - 1, 6, D - 1] = float("nan")
    lse = torch.zeros(T, Hq, device=DEV)
    out = moe().moe_kv4_attention(*attn_args(c), scale=0.1, lse=lse)
    check_poisoned(c, clean, out, lse, poisoned, 64, 0.1)


@pytest.mark.parametrize("kv", [100, 3000])
@pytest.mark.parametrize("D,qs", KERNELS)
def test_a_key_that_is_not_a_number_answers_with_none(D, qs, kv):
    """One block of one key of one head: all rows of that sequence and head see it."""
    clean = attn_case(D, 2, 4, 64, qs, [max(kv, n) for n in qs], seed=24)
    c = dict(clean, pool=clean["pool"].copy())
    T, Hq, _ = c["q"].shape
    oa.sections(c["pool"][c["table"][1, 0], 1], 64, D)[1][7, 2] = 0x7F
    poisoned = np.zeros((T, Hq), bool)
    poisoned[c["starts"][1]:c["starts"][2], 4:] = True
    lse = torch.zeros(T, Hq, device=DEV)
    out = moe().moe_kv4_attention(*attn_args(c), scale=0.1, lse=lse)
    check_poisoned(c, clean, out, lse, poisoned, 64, 0.1)


# --------------------------------------------------------- graphs and threads
@pytest.mark.parametrize("D,qs", KERNELS)
def test_a_step_in_a_graph(D, qs):
    """Pages for new tokens, norms with the write, attention, a fork, a release and a compaction, replayed on new inputs."""
    m = moe()
    B, T, Hq, Hkv, P = len(qs), sum(qs), 8, 2, 32
    M, N, S = 20, 20 * 45, len(qs) + 1
    g = torch.full((Hkv,), 5.0 / 2688, device=DEV)
    gen = torch.Generator(DEV).manual_seed(3)
    r = lambda h: torch.randn(T, h, D, generator=gen, device=DEV).bfloat16()  # noqa: E731
    q, k, v = r(Hq), r(Hkv), r(Hkv)
    a = torch.arange(900, device=DEV).unsqueeze(1) * 1e4 ** (-torch.arange(0, D, 2, device=DEV) / D)
    cs = torch.cat((a.cos(), a.sin()), 1).float().contiguous()
    offsets = dev(np.cumsum([0] + qs + [0]), I32)
    table, lens, refs = torch.full((S, M), -1, dtype=I32, device=DEV), dev([0] * S, I32), dev([0] * N, I32)
    pool = torch.zeros(1, N, Hkv, oa.record_bytes(P, D), dtype=torch.uint8, device=DEV)
    src, dst = dev([0], I32), dev([B], I32)

    def step():
        e = m.moe_kv_extend(offsets, T, table, lens, refs, P, inplace=True)
        y, _ = m.moe_qk_norm_rope(q, k, cs, e["pos"], v=v, pool=pool[0], g_k=g, g_v=g, slots=e["slots"])
        out = m.moe_kv4_attention(y, pool[0], g, g, offsets, lens, table)
        m.moe_kv_fork(src, dst, table, lens, refs, pool, P, inplace=True)
        m.moe_kv_free(dst, table, lens, refs, P, inplace=True)
        m.moe_kv_compact(table, refs, pool, inplace=True)
        return out

    fresh = [t.clone() for t in (table, lens, refs, pool)]

    def reset():
        for t, f in zip((table, lens, refs, pool), fresh):
            t.copy_(f)

    want = [step().clone() for _ in range(2)]  # the second step's context is the first one's tokens and its own
    held = [t.clone() for t in (table, lens, refs, pool)]
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    reset()
    for y in want:
        graph.replay()
        assert torch.equal(out, y)
    for t, h in zip((table, lens, refs, pool), held):
        assert torch.equal(t, h)
    assert m.moe_sync_status() == 0


def test_calls_of_several_threads():
    """Each on a stream of its own, all kernels at once."""
    m = moe()
    cases = [attn_case(D, 2, 4, 64, qs, [300] * len(qs), seed=26) for D, qs in KERNELS]
    args = [attn_args(c) for c in cases]
    want = [m.moe_kv4_attention(*a, scale=0.1) for a in args]
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(n):
        try:
            s = torch.cuda.Stream()
            for i in range(len(args)):
                j = (i + n) % len(args)
                got[n, j] = m.moe_kv4_attention(*args[j], scale=0.1, stream=s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and all(torch.equal(y, want[j]) for (_, j), y in got.items())
    assert m.moe_sync_status() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_a_key_that_is_not_a_number_is_stored_as_none(D):
    """Its blocks of 16 have scales that are not a number, all other bytes are as without it."""
    m, T, Hkv, P = moe(), 9, 3, 32
    gen = torch.Generator(DEV).manual_seed(31)
    q, k, v = (torch.randn(T, h, D, generator=gen, device=DEV).bfloat16() for h in (4, Hkv, Hkv))
    w, g = torch.ones(D, dtype=torch.bfloat16, device=DEV), torch.full((Hkv,), 0.002, device=DEV)
    slots = torch.arange(T, device=DEV) + 20

    def write():
        pool = torch.zeros(1, Hkv, oa.record_bytes(P, D), dtype=torch.uint8, device=DEV)
        m.moe_qk_norm_rope(q, k, wq=w, wk=w, v=v, pool=pool, g_k=g, g_v=g, slots=slots)
        return [s.copy() for h in range(Hkv) for s in oa.sections(pool[0, h].cpu().numpy(), P, D)]

    clean = write()
    k[4, 1, 5] = v[6, 2, 37] = float("nan")  # a norm spreads it over the head
    got = write()
    at = {(4 * 1 + 1, 24): range(D // 16), (4 * 2 + 3, 26): [2]}
    for i, (a, b) in enumerate(zip(clean, got)):
        other = np.ones(P, bool)
        for (section, token), blocks in at.items():
            if i == section:
                assert [int(x) & 0x7F for x in b[token][list(blocks)]] == [0x7F] * len(blocks)
                assert all(b[token][j] == a[token][j] for j in range(D // 16) if j not in blocks)
            if i in (section, section - 1):
                other[token] = False
        assert np.array_equal(a[other], b[other])


def test_lengths_of_a_step_are_checked():
    m = moe()
    i = lambda *s: torch.zeros(*s, dtype=I32, device=DEV)  # noqa: E731
    table, lens, refs = i(3, 2) - 1, i(3), i(8)
    for bad in (i(4), i(3).long(), torch.zeros(3, dtype=I32)):
        with pytest.raises((TypeError, ValueError), match="kv_lens"):
            m.moe_kv_extend_ex(i(4), 0, table, lens, refs, 32, out=dict(kv_lens=bad))
    with pytest.raises(ValueError, match="q_offsets"):
        m.moe_kv_extend_ex([0, 0, 0, 0], 0, table, lens, refs, 32)
    with pytest.raises(m._lib.MoEError):
        m.moe_kv_extend_ex(i(4), 0, table, lens, refs, 32, inplace=True, out=dict(kv_lens=lens))
    kv = i(3) + 9
    o = m.moe_kv_extend_ex(dev([0, 3, 3, 90], I32), 90, table, lens, refs, 32, out=dict(kv_lens=kv))  # the third has no room
    assert o["kv_lens"] is kv
    assert m.moe_sync_status() == 1 and kv.tolist() == [3, 0, 0] and o["lens"].tolist() == [3, 0, 0]


# ------------------------------------------------------------------- many forks
def test_many_forks_and_rows_named_twice():
    """More pairs than a block has threads, some with a destination that an earlier pair has named, in any order."""
    m, P, S, n = moe(), 32, 5000, 3000
    rng = np.random.default_rng(41)
    s = oa.Pages([[-1] * 3 for _ in range(S)], [0] * S, [0] * 6000, P)
    s.extend([int(x) for x in rng.integers(1, 90, 1500)] + [0] * (S - 1500))
    src, dst = rng.integers(0, 1500, n), rng.permutation(np.arange(1500, S))[:n]
    again = np.sort(rng.permutation(np.arange(1, n))[:400])
    dst[again] = dst[rng.integers(0, again)]
    dst[rng.integers(0, n, 30)] = rng.integers(-3, 1500, 30)  # in use, or none
    _, first = np.unique(dst, return_index=True)
    good = [int(i) for i in np.sort(first) if 1500 <= dst[i] < S]
    table, lens, refs = state(s)
    s.fork([int(src[i]) for i in good], [int(dst[i]) for i in good])
    same(m.moe_kv_fork(dev(src, I32), dev(dst, I32), table, lens, refs, page_size=P), s)
    assert m.moe_sync_status() == 1


def test_as_many_forks_as_a_call_takes():
    """65536 of a row of one full page.  Their check reads each pair a few times: some
    thousand steps of a block, a millisecond with a factor of five to spare."""
    m, n = moe(), 65536
    i = lambda *s: torch.zeros(*s, dtype=I32, device=DEV)  # noqa: E731
    table, lens, refs = i(n + 1, 1) - 1, i(n + 1), i(8)
    table[0], lens[0], refs[0] = 0, 32, 1
    src, dst = i(n), torch.arange(1, n + 1, dtype=I32, device=DEV)
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for _ in range(2):
        t[0].record()
        o = m.moe_kv_fork(src, dst, table, lens, refs, page_size=32)
        t[1].record()
    assert m.moe_sync_status() == 0
    assert (o["table"] == 0).all() and (o["lens"] == 32).all() and o["refs"].tolist() == [n + 1] + [0] * 7
    assert t[0].elapsed_time(t[1]) < 5
