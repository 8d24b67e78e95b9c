"""The cache class and the decoder-layer example: however a sequence's tokens
are cut into steps, forked or moved, its attention reads the same bytes."""
import os
import subprocess
import sys

import pytest
import torch

from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HQ, HKV, D, LAYERS = 8, 2, 64, 2


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def cache(rows=5, pages=40, page_size=32):
    import mixture_experts_layer_fwd_gb300 as m
    g = torch.full((LAYERS, HKV), 5.0 / 2688, device="cuda")
    return m.KV4Cache(LAYERS, pages, rows, 12, HKV, D, g, g.clone(), page_size)


def inputs(T, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda h: torch.randn(T, h, D, generator=g, device="cuda").bfloat16()  # noqa: E731
    a = torch.arange(400, device="cuda").unsqueeze(1) * 1e4 ** (-torch.arange(0, D, 2, device="cuda") / D)
    return r(HQ), r(HKV), r(HKV), torch.cat((a.cos(), a.sin()), 1).float().contiguous()


def run(c, row, rows, q, k, v, cs, cuts):
    """The tokens of one sequence in steps; outputs in order."""
    out, at = [], 0
    for n in cuts:
        c.extend([n if r == row else 0 for r in range(rows)])
        s = slice(at, at + n)
        for layer in range(LAYERS):
            y = c.attend(layer, q[s], k[s], v[s], cs)
        out.append(y)
        at += n
    return torch.cat(out)


def bytes_of(c, row, n):
    """What the cache holds of a row, in the order of its tokens."""
    pages = c.table[row, :-(-n // c.page_size)].long()
    rec, P = c.pool[:, pages], c.page_size
    cut = rec.split((P * D // 2, P * D // 16, P * D // 2, P * D // 16), -1)
    return [t.unflatten(-1, (P, -1)).transpose(1, 2).flatten(2, 3)[:, :, :n] for t in cut]


@pytest.mark.parametrize("cuts", [[200], [1] * 20 + [180], [77, 1, 1, 121], [199, 1]])
def test_steps_do_not_change_the_cache(cuts):
    import mixture_experts_layer_fwd_gb300 as m
    q, k, v, cs = inputs(200)
    a, b = cache(), cache()
    want = run(a, 0, 5, q, k, v, cs, [200])
    b.extend([0, 50, 0, 0, 0])  # pages of another row come in between
    got = run(b, 3, 5, q, k, v, cs, cuts)
    for x, y in zip(bytes_of(a, 0, 200), bytes_of(b, 3, 200)):
        assert torch.equal(x, y)
    # two roundings to bf16 of values of order one (2^-9 each) and the kernels' own 2^-10 of sum p |v| <= 4
    assert (want.float() - got.float()).abs().max() <= 2 * 2.0 ** -9 * want.float().abs().max() + 4 * 2.0 ** -10
    assert m.moe_sync_status() == 0


def test_forks_go_their_own_way_and_moving_pages_changes_nothing():
    import mixture_experts_layer_fwd_gb300 as m
    q, k, v, cs = inputs(120)
    c = cache(pages=20)
    run(c, 0, 5, q, k, v, cs, [100])
    before = bytes_of(c, 0, 100)
    c.fork([0, 0], [2, 4])
    q2, k2, v2, _ = inputs(20, seed=9)
    run(c, 2, 5, q2, k2, v2, cs, [20])
    for x, y in zip(before, bytes_of(c, 0, 100)):
        assert torch.equal(x, y)
    mine, other = bytes_of(c, 2, 120), bytes_of(c, 4, 100)
    c.free([0])
    c.compact()
    live = int((c.refs > 0).sum())
    assert (c.refs[:live] > 0).all() and int(c.table.max()) < live
    for x, y in zip(mine, bytes_of(c, 2, 120)):
        assert torch.equal(x, y)
    for x, y in zip(other, bytes_of(c, 4, 100)):
        assert torch.equal(x, y)
    assert c.lens.tolist() == [0, 0, 120, 0, 100] and m.moe_sync_status() == 0


def test_cache_reports_when_it_is_full():
    import mixture_experts_layer_fwd_gb300 as m
    c = cache(pages=2)
    c.extend([65, 0, 0, 0, 0])
    assert m.moe_sync_status() == 6 and c.lens.tolist() == [0] * 5
    with pytest.raises(ValueError, match="page_size"):
        cache(page_size=48)
    with pytest.raises(ValueError, match="extend"):
        q, k, v, cs = inputs(1)
        cache().attend(0, q, k, v, cs)


def test_decoder_layer_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_layer.py")], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "lengths [0, 136, 505, 0, 136, 0]" in r.stdout, r.stdout
