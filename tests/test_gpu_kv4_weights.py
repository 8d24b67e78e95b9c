"""Attention weights summed per key on the GPU against oracle/attention.py: ragged
batches, masks, rows that see nothing, strides, refusals, streams and graphs."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests.helpers import require_gpu, to_np_f32
from tests.test_gpu_kv4 import DEV, F32, attn_case, dev

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


def reference_lse(c, P, scale, causal, window):
    _, lse, _, _ = oa.attention(to_np_f32(c["q"]), c["pool"], c["gk"], np.ones_like(c["gk"]), c["starts"], c["lens"], c["table"],
                                scale, P, causal, window)
    return lse.astype(F32)


def call(c, P, lse, score, scale, causal=True, window=0, q=None, **kw):
    return moe().moe_kv4_weights(c["q"].to(DEV) if q is None else q, dev(c["pool"]), dev(c["gk"]), dev(lse), dev(c["starts"]),
                                 dev(c["lens"]), dev(c["table"]), score, scale=scale, causal=causal, window=window, **kw)


def check_weights(c, P, scale, causal=True, window=0, lse=None, seed=0, more=3, **kw):
    B, Hkv = len(c["lens"]), c["pool"].shape[1]
    D = c["q"].shape[2]
    rng = np.random.default_rng(seed)
    before = rng.exponential(size=(B, Hkv, c["table"].shape[1] * P + more)).astype(F32)
    lse = reference_lse(c, P, scale, causal, window) if lse is None else lse
    score = dev(before)
    out = call(c, P, lse, score, scale, causal, window, **kw)
    assert out.data_ptr() == score.data_ptr()
    got, want = score.cpu().numpy(), before.astype(np.float64)
    off = np.zeros_like(want)
    ref = oa.weights(to_np_f32(c["q"]), lse, c["pool"], c["gk"], c["starts"], c["lens"], c["table"], scale, P, causal, window)
    for b, (w, o) in enumerate(ref):
        n, L = int(c["starts"][b + 1] - c["starts"][b]), int(c["lens"][b])
        if n == 0:
            continue
        old = max(0, L - n)
        want[b, :, :old] += w[:, :old]
        want[b, :, old:L] = w[:, old:]
        rows = n * c["q"].shape[1] // Hkv
        # exponent: D / 16 instructions of 2^-22 of what they add, and a few roundings of 2^-24 of its
        # size; the exponential 2 ulp; the sums 2^-24 per row; the sum with the older one
        off[b, :, :L] = (D / 16 + 4) * 2.0 ** -22 * o + (2.0 ** -22 + rows * 2.0 ** -24) * w + 2.0 ** -24 * want[b, :, :L] + 1e-37
    bad = np.abs(got - want) > off
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], off[bad][:5])
    return score


SMALL, CHUNKS = [1, 0, 2, 1, 3], [70, 1, 0, 150, 33]


@pytest.mark.parametrize("qs", [SMALL, CHUNKS])
@pytest.mark.parametrize("D,Hkv,G,P", [(128, 2, 4, 64), (128, 1, 16, 32), (64, 2, 5, 64), (64, 1, 1, 128), (128, 1, 3, 128),
                                       (64, 3, 7, 32), (128, 5, 1, 64)])
def test_weights_of_ragged_batches(qs, D, Hkv, G, P):
    kvs = [max(n, m) for n, m in zip(qs, (P + 1, 5, 3 * P, 2 * P, 2 * P - 1))]
    check_weights(attn_case(D, Hkv, G, P, qs, kvs, seed=D + G), P, D ** -0.5)


@pytest.mark.parametrize("qs", [SMALL, CHUNKS])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 17), (True, 128), (True, 1000), (True, 2 ** 31 - 1)])
def test_weights_masks(qs, causal, window):
    kvs = [max(n, m) for n, m in zip(qs, (300, 5, 129, 260, 64))]
    check_weights(attn_case(64, 1, 4, 32, qs, kvs, seed=window % 1000), 32, 0.2, causal, window)


@pytest.mark.parametrize("qs", [[2, 1, 3, 1], [90, 40, 200, 9]])
@pytest.mark.parametrize("window", [0, 3])
def test_weights_of_rows_that_see_nothing(qs, window):
    """Fewer keys than queries: the first rows see none; no keys at all; one key."""
    check_weights(attn_case(128, 1, 2, 32, qs, [qs[0] // 2, 0, 1, qs[3]], seed=3), 32, 0.1, window=window)


@pytest.mark.parametrize("qs,kvs", [([1], [1]), ([1], [31]), ([1], [32]), ([1], [33]), ([1], [3001]), ([4], [4]), ([257], [257]),
                                    ([300], [1111])])
def test_weights_of_one_sequence(qs, kvs):
    check_weights(attn_case(128, 2, 4, 64, qs, kvs, seed=kvs[0]), 64, 128 ** -0.5)


@pytest.mark.parametrize("scale,loud", [(0.09, 12.0), (-0.09, 1.0), (0.0, 1.0), (1e-3, 300.0)])
def test_weights_scales(scale, loud):
    check_weights(attn_case(128, 1, 8, 64, [1, 30, 1], [400, 77, 513], seed=11, loud=loud), 64, scale)


@pytest.mark.parametrize("D,G,window,causal", [(64, 2, 0, True), (64, 3, 700, True), (128, 2, 0, False)])
def test_weights_of_many_rows_on_many_keys(D, G, window, causal):
    """Enough keys for items of 256 of them, rows that end inside a tile, sequences of few rows beside them."""
    qs, kvs = [150, 1, 140, 131, 129, 0, 5], [4000, 40, 4100, 3900, 3600, 9, 70]
    check_weights(attn_case(D, 8, G, 32, qs, kvs, seed=D + G), 32, D ** -0.5, causal, window)


@pytest.mark.parametrize("D,G", [(128, 16), (64, 4), (128, 4), (64, 8)])
def test_weights_of_few_rows_among_many_empty_sequences(D, G):
    """Rows that one warp holds, prepared by each block; tables of more sequences than that has room for."""
    for B, Hkv in ((1, 8), (33, 2), (130, 1), (700, 4)):
        qs, kvs = [0] * B, [(7 * b) % 90 for b in range(B)]
        qs[B // 2], kvs[B // 2] = 16 // G, 900
        if G == 4 and B > 1:
            qs[B // 2], qs[0], qs[B - 1], kvs[B - 1] = 2, 1, 1, 333
        check_weights(attn_case(D, Hkv, G, 64, qs, kvs, seed=B), 64, D ** -0.5, window=0 if B != 33 else 50)


@pytest.mark.parametrize("D,Hkv,G,qs,kvs", [(128, 4, 3, [120, 125], [4800, 5200]),   # 3 tiles of 128 rows to an item
                                            (128, 4, 2, [190, 128], [3000, 7000]),   # 3; 2
                                            (64, 4, 3, [120, 210], [6000, 3000])])   # 3; 5
def test_weights_of_items_with_an_odd_number_of_tiles(D, Hkv, G, qs, kvs):
    """Several items to a block: a slot of the rings holds tiles of either place in an item."""
    c, scale = attn_case(D, Hkv, G, 64, qs, kvs, seed=D + G), D ** -0.5
    lse = reference_lse(c, 64, scale, True, 0)
    want = check_weights(c, 64, scale, lse=lse, more=0)
    before = dev(np.random.default_rng(0).exponential(size=tuple(want.shape)).astype(F32))  # as check_weights' own
    for _ in range(20):
        assert torch.equal(call(c, 64, lse, before.clone(), scale), want)


@pytest.mark.parametrize("D,causal,window", [(128, True, 0), (64, False, 0), (64, True, 130)])
def test_weights_of_long_chunks_on_few_keys(D, causal, window):
    """Few items of many rows: their rows are split, the sums join."""
    qs, kvs = [700, 2, 513, 260], [700, 300, 600, 400]
    check_weights(attn_case(D, 1, 8, 64, qs, kvs, seed=D + window), 64, D ** -0.5, causal, window)


def test_weights_of_many_short_sequences():
    rng = np.random.default_rng(5)
    qs = [int(n) for n in rng.integers(0, 3, 330)]
    kvs = [int(n) for n in rng.integers(0, 200, 330)]
    kvs[7], qs[7], kvs[200], qs[200] = 3000, 1, 0, 2
    check_weights(attn_case(64, 2, 2, 32, qs, kvs, seed=17), 32, 0.125)


def test_a_row_with_lse_of_no_keys_gives_nothing_and_nan_goes_where_it_looks():
    c = attn_case(64, 1, 2, 32, [2, 1], [40, 50], seed=4)
    lse = reference_lse(c, 32, 0.1, True, 0)
    lse[0, 1] = -np.inf
    check_weights(c, 32, 0.1, lse=lse)
    lse[0, 0] = np.nan  # the query at place 38 of the first sequence
    before = torch.zeros(2, 1, c["table"].shape[1] * 32, device=DEV)
    s = call(c, 32, lse, before, 0.1)[:, 0]
    assert s[0, :39].isnan().all() and s[0, 39:].isfinite().all() and s[1].isfinite().all()


@pytest.mark.parametrize("qs,kvs", [([3, 1], [300, 50]), ([20, 1], [300, 50]), ([150, 1], [300, 50])])
@pytest.mark.parametrize("D", [64, 128])
def test_a_row_with_lse_of_no_keys_gives_nothing_whatever_lies_in_it(D, qs, kvs):
    """Registers, staged rows and tcgen05: a query of NaN or infinity there is as good as zeros."""
    c = attn_case(D, 1, 2, 32, qs, kvs, seed=D + qs[0])
    lse = reference_lse(c, 32, 0.1, True, 0)
    lse[qs[0] - 1], lse[1, 1], lse[qs[0], 0] = -np.inf, -np.inf, -np.inf
    q = c["q"].clone()
    want = check_weights(c, 32, 0.1, lse=lse)
    q[qs[0] - 1, 0, 5], q[qs[0] - 1, 1], q[1, 1, ::3], q[qs[0], 0] = float("nan"), float("inf"), -float("inf"), float("nan")
    assert torch.equal(check_weights(c, 32, 0.1, lse=lse, q=q.to(DEV)), want)


def test_weights_and_attention_together():
    """With the attention's own lse a query head's weights add up to one."""
    m = moe()
    for qs, kvs in (([1, 1, 3], [700, 64, 129]), ([200, 1, 90], [700, 64, 129])):
        c = attn_case(128, 2, 4, 64, qs, kvs, seed=9)
        q, T = c["q"].to(DEV), sum(qs)
        lse = torch.empty(T, 8, device=DEV)
        args = [dev(c[k]) for k in ("pool", "gk", "gv", "starts", "lens", "table")]
        m.moe_kv4_attention(q, *args, lse=lse)
        score = torch.zeros(3, 2, c["table"].shape[1] * 64, device=DEV)
        m.moe_kv4_weights(q, args[0], args[1], lse, *args[3:], score)
        # the lse is within 5e-4 of the formula's, so each weight within that part of itself
        want = torch.tensor([[n * 4.0] * 2 for n in qs], device=DEV)
        assert ((score.sum(2) - want).abs() <= 1e-3 * want).all()


def test_weights_take_slices_streams_and_graphs():
    m, c = moe(), attn_case(128, 1, 4, 64, [1, 20, 2], [200, 130, 99], seed=13)
    P, scale = 64, 0.1
    wide = torch.zeros(23, 6 * 128 + 64, dtype=torch.bfloat16, device=DEV)
    q = wide[:, 64:64 + 512].unflatten(1, (4, 128))
    q.copy_(c["q"])
    want = check_weights(c, P, scale, q=q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = check_weights(c, P, scale, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    lse = dev(reference_lse(c, P, scale, True, 0))
    args = (q, dev(c["pool"]), dev(c["gk"]), lse, dev(c["starts"]), dev(c["lens"]), dev(c["table"]))
    score = torch.zeros(3, 1, c["table"].shape[1] * P, device=DEV)
    once = m.moe_kv4_weights(*args, score.clone(), scale=scale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_kv4_weights(*args, score, scale=scale)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(score, once)
    graph.replay()
    torch.cuda.synchronize()
    old = torch.tensor([199, 110, 97], device=DEV).view(3, 1, 1) > torch.arange(score.shape[2], device=DEV)
    assert torch.equal(score, torch.where(old, once + once, once))


def test_weights_report_pages_outside_and_touch_no_other_rows():
    m, c = moe(), attn_case(64, 1, 2, 32, [1, 1], [64, 40], seed=4)
    lse = reference_lse(c, 32, 0.1, True, 0)
    c["table"][0, 1] = 99
    before = torch.full((2, 1, c["table"].shape[1] * 32), 0.5, device=DEV)
    s = call(c, 32, lse, before, 0.1)
    assert m.moe_sync_status() == 1
    assert (s[1, 0, 40:] == 0.5).all() and (s[0, 0, 64:] == 0.5).all()
    c["table"][0, 1] = 0
    c["lens"][1] = 10 ** 6  # past the table: clamped
    c["table"][1, 2:] = 0
    call(c, 32, lse, before, 0.1)
    assert m.moe_sync_status() in (0, 1)


def test_weights_refuse():
    m, c = moe(), attn_case(64, 2, 2, 32, [1, 1], [64, 40], seed=4)
    M = c["table"].shape[1]
    q, pool, gk, lse = c["q"].to(DEV), dev(c["pool"]), dev(c["gk"]), torch.zeros(2, 4, device=DEV)
    rest = (dev(c["starts"]), dev(c["lens"]), dev(c["table"]))
    score = torch.zeros(2, 2, M * 32, device=DEV)
    m.moe_kv4_weights(q[:0], pool, gk, lse[:0], *rest, score)
    assert (score == 0).all()
    for bad, error in (((q.float(), pool, gk, lse, *rest, score), TypeError), ((q, pool, gk, lse[:1], *rest, score), ValueError),
                       ((q, pool, gk, lse.double(), *rest, score), TypeError), ((q, pool, gk, lse, *rest, score[..., :M * 32 - 1].contiguous()), ValueError),
                       ((q, pool, gk, lse, *rest, score[:1]), ValueError), ((q, pool, gk, lse, *rest, score.double()), TypeError),
                       ((q, pool, gk, lse, *rest, score[..., ::2]), ValueError), ((q, pool, gk, None, *rest, score), ValueError),
                       ((q, pool, gk, lse, *rest, None), ValueError)):
        with pytest.raises(error):
            m.moe_kv4_weights(*bad)
    with pytest.raises(RuntimeError, match="INVALID"):
        m.moe_kv4_weights(q, pool, gk, lse, *rest, score, causal=False, window=4)
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        m.moe_kv4_weights(q, pool, gk, lse, *rest, score, ws=torch.empty(256, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("limit_us", [0, 5, 20])
@pytest.mark.parametrize("D,qs,kv", [(128, [300, 90, 1], 8192), (64, [500, 700, 1], 8192)])
def test_weights_that_give_up_stay_inside_their_buffers(D, qs, kv, limit_us):
    """Whatever the workspace held before; the next call is right again."""
    m, Hkv, G, P = moe(), 2, 4, 64
    T, B, Hq = sum(qs), len(qs), Hkv * G
    gen = torch.Generator(DEV).manual_seed(22)
    pool = torch.randint(0, 256, (64, Hkv, oa.record_bytes(P, D)), generator=gen, device=DEV, dtype=torch.uint8)
    pool[:, :, P * D // 2:P * D // 2 + P * D // 16] = 0x38
    g = torch.full((Hkv,), 0.01, device=DEV)
    args = (torch.randn(T, Hq, D, generator=gen, device=DEV).bfloat16(), pool, g,
            torch.full((T, Hq), 9.0, device=DEV), dev(np.cumsum([0] + qs).astype(np.int32)),
            dev(np.array([kv - 5 * i for i in range(B)], np.int32)),
            torch.randint(0, 64, (B, kv // P), generator=gen, device=DEV, dtype=torch.int32))
    want = m.moe_kv4_weights(*args, torch.zeros(B, Hkv, kv, device=DEV))
    assert torch.isfinite(want).all() and (want[0] > 0).any()
    guard = 1 << 16
    scores = torch.full((want.numel() + 2 * guard,), 3.0, device=DEV)
    size = m._lib.load().moe_kv4_weights_workspace_size(T, B, Hq, Hkv, D)
    wss = torch.full((size + 2 * guard,), 0x7F, dtype=torch.uint8, device=DEV)
    score, ws = (t[guard:t.numel() - guard] for t in (scores, wss))
    try:
        m.moe_set_wait_timeout_ns(max(1, 1000 * limit_us))
        m.moe_kv4_weights(*args, score.view(want.shape), ws=ws)
    finally:
        m.moe_set_wait_timeout_ns(0)
    assert m.moe_sync_status() in (0, 5)
    for t, v in ((scores, 3.0), (wss, 0x7F)):
        assert (t[:guard] == v).all() and (t[-guard:] == v).all()
    again = m.moe_kv4_weights(*args, torch.zeros_like(want), ws=ws)
    assert torch.equal(again, want) and m.moe_sync_status() == 0
