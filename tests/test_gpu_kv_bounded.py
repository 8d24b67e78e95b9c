"""A cache that is kept short, and steps whose drafted tokens are refused: what stays
is what was written, positions go on, forks carry their sums."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests.helpers import require_gpu, to_np_f32
from tests.test_gpu_kv_cache import D, HKV, HQ, LAYERS, bytes_of, inputs

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROWS = 5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    import mixture_experts_layer_fwd_gb300 as m
    m.moe_sync_status()
    yield
    assert m.moe_sync_status() == 0


def cache(pages=60, page_size=32, track=True):
    import mixture_experts_layer_fwd_gb300 as m
    g = torch.full((LAYERS, HKV), 5.0 / 2688, device="cuda")
    return m.KV4Cache(LAYERS, pages, ROWS, 12, HKV, D, g, g.clone(), page_size, track=track)


def step(c, counts, q, k, v, cs):
    c.extend(counts)
    return [c.attend(layer, q, k, v, cs) for layer in range(LAYERS)]


def test_tracking_changes_no_answer_and_adds_up():
    q, k, v, cs = inputs(160)
    a, b = cache(), cache(track=False)
    for lo, hi in ((0, 100), (100, 101), (101, 104), (104, 160)):
        s = slice(lo, hi)
        ya, yb = (step(c, [hi - lo, 0, 0, 0, 0], q[s], k[s], v[s], cs) for c in (a, b))
        assert all(torch.equal(x, y) for x, y in zip(ya, yb))
    # each query's heads give a weight of one each, within the lse's error
    total = a.scores[:, 0].sum(2)
    assert ((total - 160 * HQ / HKV).abs() <= 1e-3 * 160 * HQ / HKV).all()
    assert (a.scores[:, 1:] == 0).all()


@pytest.mark.parametrize("n", [150, 97])
def test_what_stays_after_eviction_is_what_attention_looked_at(n):
    q, k, v, cs = inputs(n + 40)
    c = cache()
    step(c, [0, n, 0, 40, 0], torch.cat((q[:n], q[n:])), torch.cat((k[:n], k[n:])), torch.cat((v[:n], v[n:])), cs)
    before, scores = bytes_of(c, 1, n), c.scores[:, 1].cpu().numpy()
    other = bytes_of(c, 3, 40)
    lost = c.evict(60, sinks=3, recent=20)
    assert lost.tolist() == [0, n - 60, 0, 0, 0] and c.lens.tolist() == [0, 60, 0, 40, 0]
    assert int((c.refs > 0).sum()) == 4 and c.evicted.tolist() == lost.tolist()
    after = bytes_of(c, 1, 60)
    for l in range(LAYERS):
        for h in range(HKV):
            middle = sorted(range(3, n - 20), key=lambda t: -float(scores[l, h, t]))[:60 - 23]
            stay = sorted([0, 1, 2] + middle + list(range(n - 20, n)))
            for x, y in zip(before, after):
                assert torch.equal(x[l, h, stay], y[l, h])
            assert (c.scores[l, 1, h, :60].cpu().numpy() == scores[l, h, stay]).all()
    for x, y in zip(other, bytes_of(c, 3, 40)):
        assert torch.equal(x, y)
    with pytest.raises(ValueError, match="extend"):
        c.attend(0, q[:1], k[:1], v[:1], cs)


def test_numbers_past_32_bits_evict_nothing():
    import mixture_experts_layer_fwd_gb300 as m
    q, k, v, cs = inputs(100)
    c = cache()
    step(c, [100, 0, 0, 0, 0], q, k, v, cs)
    before = bytes_of(c, 0, 100)
    for kw in (dict(keep=2 ** 32 + 8), dict(keep=2 ** 32 + 8, limit=2 ** 32 + 9, sinks=2, recent=3), dict(keep=50, limit=2 ** 40 + 60),
               dict(keep=2 ** 63, sinks=4)):
        assert c.evict(**kw).tolist() == [0] * ROWS and c.lens.tolist()[0] == 100
    for kw in (dict(keep=60, sinks=2 ** 32), dict(keep=60, recent=2 ** 32 + 1), dict(keep=-2 ** 32 + 60, limit=100),
               dict(keep=60, limit=2 ** 32 - 2 ** 33 + 80)):
        with pytest.raises(m._lib.MoEError, match="INVALID"):
            c.evict(**kw)
    for x, y in zip(before, bytes_of(c, 0, 100)):
        assert torch.equal(x, y)


def test_positions_go_on_after_eviction_and_attention_sees_what_stayed():
    import mixture_experts_layer_fwd_gb300 as m
    q, k, v, cs = inputs(130)
    c = cache()
    step(c, [100, 0, 20, 0, 0], q[:120], k[:120], v[:120], cs)
    c.evict(50, sinks=2, recent=10)
    c.extend([2, 0, 1, 0, 0])
    assert c.pos.tolist() == [100, 101, 20] and c.lens.tolist() == [52, 0, 21, 0, 0]
    y = c.attend(0, q[120:123], k[120:123], v[120:123], cs)
    qr, _ = m.moe_qk_norm_rope(q[120:123], k[120:123], cs, c.pos)
    pool = c.pool[0].cpu().numpy()
    ref, _, weight, all_v = oa.attention(to_np_f32(qr), pool, c.g_k[0].cpu().numpy(), c.g_v[0].cpu().numpy(), [0, 2, 2, 3, 3, 3],
                                         [52, 0, 21, 0, 0], c.table.cpu().numpy(), D ** -0.5, 32)
    # as for attention: bf16's rounding, P in fp16 and the scores' sums
    assert (np.abs(to_np_f32(y) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * weight + 2.0 ** -32 * all_v).all()
    c.free([0])
    c.extend([1, 0, 0, 0, 0])
    assert c.pos.tolist() == [0]  # a row that became empty begins anew


def test_refused_tokens_leave_no_trace():
    """Steps of drafts, some of them refused, leave the bytes of the accepted tokens alone."""
    rng = np.random.default_rng(1)
    V = 50
    q, k, v, cs = inputs(400)
    a, b = cache(track=False), cache(track=False)
    at = [60, 33, 0, 64, 95]
    first = sum(at)
    for c in (a, b):
        step(c, at, q[:first], k[:first], v[:first], cs)
    where = first
    for _ in range(4):
        counts = [int(x) for x in rng.integers(1, 5, ROWS)]
        counts[2] = 0
        T = sum(counts)
        s = slice(where, where + T)
        where += T
        step(a, counts, q[s], k[s], v[s], cs)
        r = a.verify(torch.randn(T, V, device="cuda"), torch.from_numpy(rng.integers(0, V, T).astype(np.int32)).cuda(),
                     torch.rand(T, device="cuda") * 0.05, torch.rand(ROWS, device="cuda"))
        took = [int(x) + 1 if n else 0 for x, n in zip(r["accepted"], counts)]
        assert [int(x) for x in r["refused"]] == [n - m for n, m in zip(counts, took)]
        starts = np.cumsum([s.start] + counts)
        rows = [t for i in range(ROWS) for t in range(starts[i], starts[i] + took[i])]
        step(b, took, q[rows], k[rows], v[rows], cs)
        assert a.lens.tolist() == b.lens.tolist()
    for row, n in enumerate(a.lens.tolist()):
        for x, y in zip(bytes_of(a, row, n), bytes_of(b, row, n)):
            assert torch.equal(x, y)
    assert sorted(a.refs.tolist()) == sorted(b.refs.tolist())


@pytest.mark.parametrize("by_hand", [False, True])
def test_refused_tokens_leave_no_trace_in_the_sums(by_hand):
    """The sums are those of a cache that only ever saw the accepted tokens, and add up to one per
    query and head of these; whether verify() or the caller's own drop() refuses."""
    rng = np.random.default_rng(2)
    V = 50
    q, k, v, cs = inputs(400)
    a, b = cache(), cache()
    at = [60, 33, 0, 64, 95]
    first = sum(at)
    for c in (a, b):
        step(c, at, q[:first], k[:first], v[:first], cs)
    where, dropped = first, 0
    for _ in range(6):
        counts = [int(x) for x in rng.integers(1, 6, ROWS)]
        counts[2] = 0
        T = sum(counts)
        s = slice(where, where + T)
        where += T
        step(a, counts, q[s], k[s], v[s], cs)
        if by_hand:
            refused = [int(rng.integers(0, max(1, n))) for n in counts]
            a.drop(refused)
        else:
            refused = a.verify(torch.randn(T, V, device="cuda"), torch.from_numpy(rng.integers(0, V, T).astype(np.int32)).cuda(),
                               torch.rand(T, device="cuda") * 0.05, torch.rand(ROWS, device="cuda"))["refused"].tolist()
        dropped += sum(refused)
        took = [n - r for n, r in zip(counts, refused)]
        starts = np.cumsum([s.start] + counts)
        rows = [t for i in range(ROWS) for t in range(starts[i], starts[i] + took[i])]
        step(b, took, q[rows], k[rows], v[rows], cs)
        assert a.lens.tolist() == b.lens.tolist()
    assert dropped > 20
    for row, n in enumerate(a.lens.tolist()):
        x, y = a.scores[:, row, :, :n], b.scores[:, row, :, :n]
        # each attention's lse is within 5e-4 of the formula's, and so is every weight
        assert ((x - y).abs() <= 1.1e-3 * y).all()
        assert ((x.sum(2) - n * HQ / HKV).abs() <= 1e-3 * n * HQ / HKV).all()


def test_sums_wait_for_the_end_of_a_step():
    q, k, v, cs = inputs(130)
    a, b, c = cache(), cache(), cache()
    for s, counts in ((slice(0, 100), [60, 0, 40, 0, 0]), (slice(100, 108), [5, 0, 3, 0, 0])):
        step(a, counts, q[s], k[s], v[s], cs)
        step(b, counts, q[s], k[s], v[s], cs)
        b.scores  # reading takes in what waits
        c.extend(counts, final=True)
        for layer in range(LAYERS):
            c.attend(layer, q[s], k[s], v[s], cs)
        assert not c._waiting
    assert len(a._waiting) == LAYERS and not b._waiting
    assert torch.equal(a.scores, b.scores) and torch.equal(a.scores, c.scores) and not a._waiting
    # whatever ends the step takes them in first; rows and pages as attention had them
    for end in (lambda x: x.extend([1] + [0] * 4), lambda x: x.free([0]), lambda x: x.compact(), lambda x: x.fork([0], [1]),
                lambda x: x.evict(20, sinks=2, recent=5)):
        one, two = cache(), cache()
        for x in (one, two):
            step(x, [60, 0, 40, 0, 0], q[:100], k[:100], v[:100], cs)
            step(x, [5, 0, 3, 0, 0], q[100:108], k[100:108], v[100:108], cs)
        two.scores
        end(one), end(two)
        assert torch.equal(one._scores, two._scores) and not one._waiting
    # a layer once more: its first sums are taken in
    c.extend([1] + [0] * 4)
    for _ in range(2):
        c.attend(0, q[108:109], k[108:109], v[108:109], cs)
    assert len(c._waiting) == 1
    old = a.scores[0, 0, :, :65].sum()
    assert abs(float(c.scores[0, 0, :, :66].sum() - old) - 2 * HQ) <= 0.05 * 2 * HQ
    c.extend([1] + [0] * 4, final=True)
    with pytest.raises(ValueError, match="final"):
        c.verify(torch.zeros(1, 4, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda"),
                 torch.zeros(ROWS, device="cuda"))
    for bad in ([1, 2], torch.zeros(4, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError, match="counts"):
            c.drop(bad)
    assert c.q_offsets is not None


def test_sums_of_another_stream_and_of_a_graph():
    q, k, v, cs = inputs(80)
    a, b = cache(), cache()
    for c in (a, b):
        step(c, [70, 0, 0, 0, 0], q[:70], k[:70], v[:70], cs)
    base = a.scores.clone()
    assert torch.equal(base, b.scores)
    side = torch.cuda.Stream()
    step(a, [2, 0, 0, 0, 0], q[70:72], k[70:72], v[70:72], cs)
    b.extend([2, 0, 0, 0, 0])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for layer in range(LAYERS):
            b.attend(layer, q[70:72], k[70:72], v[70:72], cs)
    torch.cuda.current_stream().wait_stream(side)
    a.drop([1, 0, 0, 0, 0]), b.drop([1, 0, 0, 0, 0])
    assert torch.equal(a.scores[:, :, :, :71], b.scores[:, :, :, :71])
    # a replay adds the weights of its step each time
    before = a.scores.clone()
    a.extend([1, 0, 0, 0, 0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for layer in range(LAYERS):
            a.attend(layer, q[72:73], k[72:73], v[72:73], cs)
    assert not a._waiting
    for n in (1, 2):
        graph.replay()
        gave = a.scores[:, 0, :, :71] - before[:, 0, :, :71]
        last = a.scores[:, 0, :, 71]
        assert ((gave.sum(2) / n + last - HQ / HKV).abs() <= 2e-3 * HQ / HKV).all()
    # sums that wait are not caught by a capture
    b.extend([1, 0, 0, 0, 0])
    b.attend(0, q[72:73], k[72:73], v[72:73], cs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(ValueError, match="capture"):
        with torch.cuda.graph(graph):
            b.evict(40)
    assert len(b._waiting) == 1
    torch.cuda.synchronize()
    b.evict(40)
    assert b.lens.tolist() == [40, 0, 0, 0, 0]


def test_rows_that_found_no_room_lose_nothing():
    import mixture_experts_layer_fwd_gb300 as m
    q, k, v, cs = inputs(200)
    c = cache(pages=4, track=False)
    step(c, [60, 62, 0, 0, 0], q[:122], k[:122], v[:122], cs)
    step(c, [4, 4, 0, 0, 0], q[122:130], k[122:130], v[122:130], cs)  # the second row finds no third page
    assert m.moe_sync_status() == 6 and c.lens.tolist() == [64, 62, 0, 0, 0]
    r = c.verify(torch.zeros(8, 9, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda"), torch.full((8,), 0.99, device="cuda"),
                 torch.zeros(ROWS, device="cuda"))
    assert r["refused"].tolist()[:2] == [3, 3] and c.lens.tolist() == [61, 62, 0, 0, 0]


def test_forks_carry_their_sums_and_go_their_own_way():
    q, k, v, cs = inputs(150)
    c = cache()
    step(c, [120, 10, 0, 0, 0], q[:130], k[:130], v[:130], cs)
    c.evict(100, sinks=1, recent=9)
    c.fork([0, 1, 0], [2, 4, 4])  # row 4 is named twice: the first pair has it
    import mixture_experts_layer_fwd_gb300 as m
    assert m.moe_sync_status() == 1
    assert c.evicted.tolist() == [20, 0, 20, 0, 0] and c.lens.tolist() == [100, 10, 100, 0, 10]
    assert torch.equal(c.scores[:, 2, :, :100], c.scores[:, 0, :, :100]) and torch.equal(c.scores[:, 4, :, :10], c.scores[:, 1, :, :10])
    c.fork([1], [2])  # not empty: it keeps what it has
    assert m.moe_sync_status() == 1 and c.evicted.tolist()[2] == 20
    assert torch.equal(c.scores[:, 2, :, :100], c.scores[:, 0, :, :100])
    kept = bytes_of(c, 0, 100)
    step(c, [0, 0, 1, 0, 0], q[130:131], k[130:131], v[130:131], cs)
    assert c.pos.tolist() == [120]
    c.evict(40, limit=100, sinks=1, recent=9)  # row 2 alone is past the limit
    assert c.lens.tolist() == [100, 10, 40, 0, 10]
    for x, y in zip(kept, bytes_of(c, 0, 100)):
        assert torch.equal(x, y)


def test_a_fork_that_finds_no_page_counts_positions_from_0():
    import mixture_experts_layer_fwd_gb300 as m
    q, k, v, cs = inputs(220)
    c = cache(pages=4)
    step(c, [120, 0, 0, 0, 0], q[:120], k[:120], v[:120], cs)
    c.evict(20, sinks=1, recent=9)
    step(c, [0, 0, 96, 0, 0], q[120:216], k[120:216], v[120:216], cs)
    c.fork([0], [1])
    assert m.moe_sync_status() == 6 and c.lens.tolist() == [20, 0, 96, 0, 0] and c.evicted.tolist() == [100, 0, 0, 0, 0]
    c.free([2])
    step(c, [1, 3, 0, 0, 0], q[216:], k[216:], v[216:], cs)
    assert c.pos.tolist() == [120, 0, 1, 2]


def test_pages_past_four_gigabytes():
    """Weights, eviction and roll-back of a sequence on the last pages of a pool are those on its first."""
    import mixture_experts_layer_fwd_gb300 as m
    P, H, head, N, M = 64, 2, 128, 240000, 10
    gen = torch.Generator("cuda").manual_seed(31)
    pool = torch.empty(1, N, H, oa.record_bytes(P, head), dtype=torch.uint8, device="cuda")
    pool[:, :M] = torch.randint(0, 256, pool[:, :M].shape, generator=gen, device="cuda", dtype=torch.uint8)
    for at in (P * head // 2, P * head // 16 * 9 + P * head // 2):
        pool[:, :M, :, at:at + P * head // 16] &= 0x3F
    pool[:, N - M:] = pool[:, :M]
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.stack((torch.arange(M), torch.arange(N - M, N))).to(**i32)
    refs = torch.zeros(N, **i32)
    refs[table.flatten().long()] = 1
    lens = torch.tensor([M * P - 7] * 2, **i32)
    g = torch.full((H,), 0.02, device="cuda")
    for n in (1, 40):  # registers, tcgen05
        q = torch.randn(n, 4 * H, head, generator=gen, device="cuda").bfloat16().repeat(2, 1, 1)
        off = torch.tensor([0, n, 2 * n], **i32)
        lse = torch.empty(2 * n, 4 * H, device="cuda")
        m.moe_kv4_attention(q, pool[0], g, g, off, lens, table, lse=lse)
        score = m.moe_kv4_weights(q, pool[0], g, lse, off, lens, table, torch.zeros(2, H, M * P, device="cuda"))
        assert torch.equal(score[0], score[1]) and (score[0, :, :M * P - 7] > 0).any()
    r = m.moe_kv4_evict(table, lens, refs, pool, score[None].contiguous(), 300, sinks=3, recent=50, D=head, inplace=True)
    assert r["lens"].tolist() == [300, 300] and r["table"][1, :5].tolist() == list(range(N - M, N - M + 5))
    assert torch.equal(pool[:, :4], pool[:, N - M:N - M + 4]) and (r["table"][:, 5:] == -1).all()
    r = m.moe_kv_drop(torch.tensor([1, 299], **i32), r["table"], r["lens"], r["refs"], pool, P, inplace=True)
    assert r["lens"].tolist() == [299, 1] and int(r["refs"].sum()) == 6


def test_a_window_of_first_and_last_tokens_needs_no_tracking():
    q, k, v, cs = inputs(120)
    c = cache(track=False)
    step(c, [120, 0, 0, 0, 0], q, k, v, cs)
    before = bytes_of(c, 0, 120)
    c.evict(40, sinks=4, recent=36)
    for x, y in zip(before, bytes_of(c, 0, 40)):
        assert torch.equal(torch.cat((x[:, :, :4], x[:, :, 84:]), 2), y)
    with pytest.raises(ValueError, match="track"):
        c.evict(40, sinks=4, recent=30)
    with pytest.raises(ValueError, match="verify"):
        c.verify(torch.zeros(1, 4, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda"),
                 torch.zeros(ROWS, device="cuda"))


@pytest.mark.parametrize("T", [1, 32, 33, 200])
def test_a_quantised_matrix_takes_any_number_of_tokens(T):
    import mixture_experts_layer_fwd_gb300 as m
    g = torch.Generator("cuda").manual_seed(T)
    w = m.quantize_weights((torch.randn(96, 256, generator=g, device="cuda") / 16).bfloat16())
    x, add = (torch.randn(T, n, generator=g, device="cuda").bfloat16() for n in (256, 96))
    from oracle import nvfp4
    wd = nvfp4.dequantize(w.codes.cpu().numpy(), w.sf.cpu().numpy(), w.g.cpu().numpy()[0])
    want = to_np_f32(x).astype(np.float64) @ wd.T
    size = np.abs(to_np_f32(x)) @ np.abs(wd).T
    got, plus = to_np_f32(w.linear(x)), to_np_f32(w.linear(x, add=add))
    # bf16's half step, sums of 256 products in fp32; with the sum another rounding
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -14 * size).all()
    a = to_np_f32(add).astype(np.float64)
    assert (np.abs(plus - want - a) <= 2.0 ** -8 * (np.abs(want) + np.abs(want + a)) + 2.0 ** -13 * size).all()
    assert w.linear(x, out_dtype=torch.float32).dtype == torch.float32


@pytest.mark.parametrize("rows,cols", [(96, 256), (50, 96), (40, 320)])
def test_a_quantised_matrix_gives_fp32_sums_for_any_number_of_tokens(rows, cols):
    """What is asked for in fp32 is not rounded to bf16 on the way, whatever the matrix's size:
    a token's outputs are those that it has alone among up to 32."""
    import mixture_experts_layer_fwd_gb300 as m
    from oracle import nvfp4
    g = torch.Generator("cuda").manual_seed(rows)
    w = m.quantize_weights((torch.randn(rows, cols, generator=g, device="cuda") / 16).bfloat16())
    wd = nvfp4.dequantize(w.codes.cpu().numpy(), w.sf.cpu().numpy(), w.g.cpu().numpy()[0])
    x, add = (torch.randn(77, n, generator=g, device="cuda").bfloat16() for n in (cols, rows))
    y, size = to_np_f32(x).astype(np.float64) @ wd.T, np.abs(to_np_f32(x)) @ np.abs(wd).T
    for T in (32, 33, 64, 77):
        for a in (None, add[:T]):
            got = w.linear(x[:T], add=a, out_dtype=torch.float32)
            want = y[:T] + (0 if a is None else to_np_f32(a))
            # cols / 16 instructions and 16 parts, 2^-22 of the sum of magnitudes each; the one rounding
            off = (cols / 16 + 16) * 2.0 ** -22 * size[:T] + 2.0 ** -23 * np.abs(want)
            assert got.dtype == torch.float32 and got.shape == (T, rows)
            assert (np.abs(to_np_f32(got) - want) <= off).all()
            assert w.linear(x[:T], add=a).dtype == torch.bfloat16
    wide = torch.zeros(40, cols + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:] = x[:40]
    assert torch.equal(w.linear(wide[:, 8:], out_dtype=torch.float32), w.linear(x[:40], out_dtype=torch.float32))
    for bad in (add[:50], add):
        with pytest.raises(ValueError):
            w.linear(x[:64], add=bad, out_dtype=torch.float32)


@pytest.mark.parametrize("T", [1, 7, 40])
def test_a_quantised_matrix_takes_tokens_wherever_they_lie(T):
    import mixture_experts_layer_fwd_gb300 as m
    g = torch.Generator("cuda").manual_seed(3)
    w = m.quantize_weights((torch.randn(96, 256, generator=g, device="cuda") / 16).bfloat16())
    x = torch.randn(T, 256, generator=g, device="cuda").bfloat16()
    want = [w.linear(x), w.linear(x, out_dtype=torch.float32)]
    for more, at in ((4, 0), (8, 4), (3, 1)):
        wide = torch.zeros(T, 256 + more, dtype=torch.bfloat16, device="cuda")
        wide[:, at:at + 256] = x
        y = wide[:, at:at + 256]
        assert torch.equal(w.linear(y), want[0]) and torch.equal(w.linear(y, out_dtype=torch.float32), want[1])


def test_speculative_decoding_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "speculative_decoding.py")], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "drafts taken" in r.stdout, r.stdout
